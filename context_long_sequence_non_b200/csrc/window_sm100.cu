// window_sm100.cu -- windowed attention on B200 tensor cores (tcgen05 + TMEM + TMA), bf16 in.
//
// For every (b, h, query row i) at position p the softmax runs over the keys of two ranges, the
// early (sink) keys [0, early) and the window [lo, hi) (window.h), streamed over 64-key blocks:
//   S = Q K^T,  x = S scale log2(e),  m' = max(m, x),  O' = O 2^(m - m') + 2^(x - m') V,
// with the same base-2 online softmax and reference-max rule as attn_sm100.cu: a row's reference
// moves only when a key above it could carry 1/kMinorWeightInv of the row or exceeds it by
// rescale_log2, so that most blocks rescale nothing.
//
// One CTA takes 128 query rows -- tokens of one (b, h), or fewer tokens of 2, 4, .. heads that share a
// key head -- and two CTAs share an SM.  Windows are short -- twenty to seventy
// blocks -- so a CTA's start (barriers, TMEM, the first loads) and its epilogue
// would be a large share of its life if nothing ran beside them; with two independent CTAs one's
// softmax, start and end overlap the other's matrix products, and a tile visits its own key
// blocks and no neighbour's.  The price, K and V not shared between two query tiles, is L2
// traffic of 32 KB per 128 x 64 products, under half of what L2 delivers.  Blocks start at the
// first key that the tile sees, not at a multiple of 64: a window of 4096 costs 66 of them.
//   warps 0-3  softmax, one thread per query row = TMEM lane
//   warp  4    TMA producer: Q, then per block K into one ring and V into another; the first
//              loads leave before the CTA's warps have met
//   warp  5    TMEM allocator; clears V rows that no row of the tile sees (below); one of its
//              threads issues every tcgen05.mma
// TMEM (256 columns): two S buffers of 64 fp32 (P written back over them as bf16 pairs) | O (D
// fp32).  With two, S of block j + 1 is computed while the softmax of block j runs, and only P V
// stands between a handoff and the S after next.  One buffer of 128 keys, S behind P V, took 3 to 8%
// longer on every case although its products are wider (N = 64 runs at about 70% of the N = 128
// rate): each block then paid a wake-up, P V and Q K^T between two softmaxes.
// A bf16 result leaves through shared memory and one TMA store a tile; fp32 and merged ones through
// shared memory and whole rows a warp, the running O's loads issued before the last product
// is done (one 64-key block merged into 256 x 2 heads in fp32: 6.3 us; 9.1 with each thread on its
// own row).
//
// Few tiles.  Where they leave SMs idle, a cluster of 2, 4 or 8 CTAs shares the key blocks of a tile
// and folds its parts (m, l, O) through distributed shared memory, each CTA 128 / n rows, in a fixed
// order (plan below): 8 tiles of 1540 keys 20 -> 8.4 us, 76 tiles of 2400 29 -> 19.
//
// What bounds it.  64 keys cost a softmax warp 1475 cycles with its neighbour on the same scheduler:
// 850 in the exponentials (512 of them the special-function unit's), 220 from S to the row maximum,
// 100 for P's stores, 300 to the next S; the tensor pipe is busy about 60% of the time.  Moving a
// share of the exponentials to the FMA pipe (1, 2 or 3 of 8, a polynomial) changes nothing.  At the
// large sizes the card is at its power cap besides (1.4 to 1.55 GHz).  Measured: 44160 tokens x
// 16 heads, causal window 4096 with 64 sinks, 1.41 to 1.49 ms = 962 to 1017 TFLOP/s of visible products
// (heads of 64: 1.05 ms = 684); 4608 x 24, 512 to either side with 512 sinks, 97 us = 815 (heads of 64: 75 us
// = 525).  More softmax warps are not what is missing: the dense kernel (attn_sm100.cu) has as many an SM
// and the same exponentials, and takes 13.2 ms where this one takes 17.0 on 44160 x 16 heads without bounds.
// It has N = 128 products, hands P over in halves, and 216 registers a softmax thread.
// Tried and not kept, on the
// 128-key form: two 128-row tiles in one CTA with shared K and V, one CTA per item (2% slower on
// the first case, 40% at 333 rows) and persistent over items (19% slower).
//
// Hidden keys.  A block is masked per element only where some row of the tile does not see all of
// it, and a hidden key's weight is exactly 0.  0 x NaN is NaN, though, so V rows that no row of the
// tile sees (past a sequence's length, outside the window) are cleared in shared memory before the
// product.
// Every wait is bounded (mbar_wait): a stalled pipeline sets the device error word and the CTA
// drains and exits.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "window.h"

namespace cpattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlockM = 128;
constexpr int kBlockN = 64;
// Six warps: two CTAs per SM then have 168 registers a thread (a 224-thread CTA would have 144, a
// 256-thread one 128).  Writing forms use 115 to 119 of them, merging ones 123 to 163; merging into fp32 at D = 128, whose threads
// hold 16 vectors of the running O beside a row's 64 logits, spills 24 bytes.
constexpr int kThreads = 192;
constexpr int kWarpProducer = 4, kWarpMma = 5;
constexpr uint32_t kTmemCols = 256;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMinorWeightInv = 8;   // see attn_sm100.cu
constexpr int kPairs = kBlockN / 2;
constexpr int kMaxCluster = 8;

template <int D>
struct Geometry {
  static constexpr int kBoxes = D / 64;                 // 64-column (128-byte) boxes per row
  static constexpr int kQBoxBytes = kBlockM * 128;      // a box of 128 query rows
  static constexpr int kBoxBytes = kBlockN * 128;       // a box of 64 keys
  static constexpr int kQBytes = kBoxes * kQBoxBytes;
  static constexpr int kTileBytes = kBoxes * kBoxBytes; // K or V of a block
  // K and V blocks in flight: what two CTAs per SM leave room for
  static constexpr int kK = D == 128 ? 2 : 4;
  static constexpr int kV = D == 128 ? 3 : 4;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kK * kTileBytes;
  static constexpr int kOffBars = kOffV + kV * kTileBytes;
  static constexpr int kSmem = kOffBars + 256;
  static constexpr int kOffParts = kBlockM * D * 4;  // behind a staged O: its rows' m and l
  static_assert(kOffParts + kBlockM * 8 <= kOffBars);
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  // A third would wait on its SM for TMEM that a CTA of another cluster holds while that cluster waits
  // for a CTA behind it.
  static_assert(3 * (kSmem + 1024) > 228 * 1024, "no more than two CTAs per SM");
};

struct __align__(8) Barriers {
  uint64_t q_full, o_full, drain, pv_done;
  uint64_t s_full[2], p_full[2];  // of the S buffer that block j uses, j & 1
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Barriers) <= 256, "barrier block");

// The key blocks of one tile: n_early blocks from key 0, then blocks from key w0.
struct Blocks {
  int early, lo, hi;  // keys that some row of the tile sees: [0, early) and [lo, hi)
  int n_early, w0;
  int first, n;  // this block's share of them: n from block `first` on
  __device__ __forceinline__ int base(int j) const {
    j += first;
    return j < n_early ? j * kBlockN : w0 + (j - n_early) * kBlockN;
  }
  // does some row of the tile see every key of [k0, k1)?
  __device__ __forceinline__ bool all_seen(int k0, int k1) const {
    return k1 <= early || (k0 >= lo && k1 <= hi);
  }
};

__device__ __forceinline__ Blocks tile_blocks(const WindowCall& c, int p_first, int p_last, int len, int rank,
                                              int n_ranks) {
  const KeyRange a = visible_keys(p_first, c.left, c.right, c.sinks, len);
  const KeyRange z = visible_keys(p_last, c.left, c.right, c.sinks, len);
  Blocks t;
  t.hi = z.hi;
  t.lo = a.lo < t.hi ? a.lo : t.hi;
  t.early = c.sinks < t.hi ? c.sinks : t.hi;
  if (t.early >= t.lo) t.early = 0, t.lo = 0;  // one range
  t.n_early = (t.early + kBlockN - 1) / kBlockN;
  t.w0 = t.lo > t.n_early * kBlockN ? t.lo : t.n_early * kBlockN;
  const int all = t.n_early + (t.hi > t.w0 ? (t.hi - t.w0 + kBlockN - 1) / kBlockN : 0);
  t.first = 0;
  t.n = all;
  if (n_ranks > 1) {
    const int share = (all + n_ranks - 1) / n_ranks;
    t.first = min(rank * share, all);
    t.n = min(share, all - t.first);
  }
  return t;
}

// 4-D tiled tensor store shared -> global, and the wait until the shared memory has been read.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// the low n bits, n clamped to 0..32
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// The rows of a tile: 2^lg heads that share a key head, and 128 / 2^lg tokens.
struct Rows {
  int first, b, h0, lg;  // row 0 is token `first` of head h0
  __device__ __forceinline__ int token(int r) const { return first + (r >> lg); }
  __device__ __forceinline__ int head(int r) const { return h0 + (r & ((1 << lg) - 1)); }
  // the row's place among the D-element rows of a packed [B][Sq][H][D] tensor, from row 0's on
  __device__ __forceinline__ size_t base(const WindowCall& c) const { return (size_t(b) * c.Sq + first) * c.H + h0; }
  __device__ __forceinline__ unsigned place(const WindowCall& c, int r) const {
    return unsigned(r + (r >> lg) * (c.H - (1 << lg)));
  }
  // its LSE (of the last token past the end)
  __device__ __forceinline__ size_t lse(const WindowCall& c, int r) const {
    return (size_t(b) * c.H + head(r)) * c.Sq + min(token(r), c.Sq - 1);
  }
};

// What becomes of a tile's result.
enum Result : int {
  kWrite = 0,       // written
  kMerge = 1,       // merged into the running (out, lse) in place
  kMergeFrom32 = 2  // merged with the running (o_run fp32, lse) into bf16 out
};

// What a row's sum over keys (reference m in units of log2, sum l) and, merging, the running row
// (log-sum-exp la) come to: O = fa running + fc new.  l is 0 for a row that saw no key and 1 or more for
// one that did; m does not tell them apart, since it is -inf for NaN scores too (maxima drop them), whose
// NaN l and O are the result.
struct RowEnd {
  float fa, fc, lse;
  bool write;
};

template <int kResult>
__device__ __forceinline__ RowEnd finish_row(float m, float l, float la, bool in_range) {
  const bool empty = l == 0.f;
  const float lc2 = m + log2f(l);
  RowEnd r{0.f, empty ? 0.f : 1.0f / l, empty ? -INFINITY : lc2 * kLn2, in_range};
  if constexpr (kResult != kWrite) {
    if (kResult == kMerge && empty) r.write = false;  // nothing to add: the running row stays as it is
    if (empty) {  // the running row alone, rounded (0 when it is empty too)
      r.fa = la == -INFINITY ? 0.f : 1.f;
      r.lse = la;
    } else {
      const float la2 = la * kLog2e;
      const float mx = fmaxf(la2, lc2);
      const float wa = exp2f(la2 - mx), wc = exp2f(lc2 - mx);
      const float tot = wa + wc;
      r.fa = wa / tot;
      r.fc = wc / (tot * l);
      r.lse = (mx + log2f(tot)) * kLn2;
    }
  }
  return r;
}

// The rows of a tile that one of its N blocks finishes: parts (m, l, O), each in its block's shared
// memory, added in the order of the parts.  16 remote reads of 16 bytes a lane are in flight.
template <int D, bool kOutF32, int kResult, int N>
__device__ __forceinline__ void fold_parts(const WindowCall& c, const cg::cluster_group& cluster, uint8_t* smem,
                                           const Rows& rows) {
  constexpr bool kAcc = kResult != kWrite;
  constexpr int kShare = kBlockM / N / 4;  // rows of a warp
  constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes, kRows = 16 / N;  // of a row; of an instruction; in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (int(cluster.block_rank()) * 4 + warp) * kShare;
  float* ml = reinterpret_cast<float*>(smem + Geometry<D>::kOffParts);
  float w[N], l = 0.f, la = 0.f, m = -INFINITY;  // of row r0 + lane
  const int mine = r0 + min(lane, kShare - 1);
  const bool in_range = rows.token(mine) < c.Sq;
  const size_t lse_idx = rows.lse(c, mine);
  const unsigned place = in_range ? rows.place(c, mine) : 0u;  // past the end any row may be read
  if (kAcc) la = c.lse[lse_idx];
  float lk[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    w[k] = *cluster.map_shared_rank(ml + mine, k);
    lk[k] = *cluster.map_shared_rank(ml + kBlockM + mine, k);
  }
  const int sub = lane / kLanes, vec = lane % kLanes;
  const size_t out_base = rows.base(c) * D + 4 * vec;
  RowEnd end;
#pragma unroll
  for (int s0 = 0; s0 < kShare / kAtOnce; s0 += kRows) {
    float4 x[kRows][N], run[kAcc ? kRows : 1];
#pragma unroll
    for (int s = 0; s < kRows; ++s) {
      if (s0 + s >= kShare / kAtOnce) continue;
      const int r = r0 + kAtOnce * (s0 + s) + sub;
      float4* part = reinterpret_cast<float4*>(smem) + r * (D / 4) + (vec ^ (r & 7));
#pragma unroll
      for (int k = 0; k < N; ++k) x[s][k] = *cluster.map_shared_rank(part, k);
      if constexpr (kAcc) {
        const size_t at = out_base + size_t(__shfl_sync(0xffffffffu, place, kAtOnce * (s0 + s) + sub)) * D;
        if constexpr (kResult == kMergeFrom32) {
          run[s] = *reinterpret_cast<const float4*>(c.o_run + at);
        } else if constexpr (kOutF32) {
          run[s] = *reinterpret_cast<const float4*>(static_cast<const float*>(c.out) + at);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(c.out) + at);
          run[s] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        }
      }
    }
    if (s0 == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) m = fmaxf(m, w[k]);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        w[k] = lk[k] == 0.f ? 0.f : ex2(w[k] - m);  // 0: that part saw no key
        l = fmaf(w[k], lk[k], l);
      }
      end = finish_row<kResult>(m, l, la, in_range);
#pragma unroll
      for (int k = 0; k < N; ++k) w[k] *= end.fc;
      if (lane < kShare && end.write && c.lse != nullptr) c.lse[lse_idx] = end.lse;
    }
#pragma unroll
    for (int s = 0; s < kRows; ++s) {
      if (s0 + s >= kShare / kAtOnce) continue;
      const int i = kAtOnce * (s0 + s) + sub;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (kAcc) {
        const float f = __shfl_sync(0xffffffffu, end.fa, i);
        if (f != 0.f)  // an empty running row may hold anything
          o = make_float4(f * run[s].x, f * run[s].y, f * run[s].z, f * run[s].w);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w[k], i);
        o.x = fmaf(wk, x[s][k].x, o.x), o.y = fmaf(wk, x[s][k].y, o.y);
        o.z = fmaf(wk, x[s][k].z, o.z), o.w = fmaf(wk, x[s][k].w, o.w);
      }
      const int live = __shfl_sync(0xffffffffu, int(end.write), i);
      const size_t at = out_base + size_t(__shfl_sync(0xffffffffu, place, i)) * D;
      if (live) {
        if constexpr (kOutF32) *reinterpret_cast<float4*>(static_cast<float*>(c.out) + at) = o;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.out) + at) =
              make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      }
    }
  }
}

template <int D, bool kOutF32, int kResult, bool kSplit>
__global__ void __launch_bounds__(kThreads, 2)
    window_sm100_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowCall c,
                        const __grid_constant__ CUtensorMap tm_o, int lg, float scale_log2, float rescale_log2,
                        int* err, long long wait_limit) {
  using G = Geometry<D>;
  constexpr bool kAcc = kResult != kWrite;
  extern __shared__ __align__(1024) uint8_t smem[];
  Barriers& bars = *reinterpret_cast<Barriers*>(smem + G::kOffBars);
  const uint32_t smem_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // CTAs run in index order: the tiles with the most keys (the last ones, when the window grows with
  // the position) come first, those of all heads beside one another, so that the grid as a whole ends
  // on short ones.  Head by head instead it ends on the last head's full range: causal 8192 x 16 heads
  // 302 us against 264, a ring step's 5520 rows x 16 heads in 3 parts 385 against 357, 4608 x 24 103
  // against 100; 44160 x 16, where a head alone fills the GPU, 1450 against 1462
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = kSplit ? int(cluster.block_rank()) : 0, n_ranks = kSplit ? int(cluster.num_blocks()) : 1;
  const unsigned n_heads = unsigned(c.H >> lg) * unsigned(c.B), item = blockIdx.x / unsigned(n_ranks);
  const int tile = int((gridDim.x / unsigned(n_ranks) - 1 - item) / n_heads);
  const int bh = int(item % n_heads);
  const int b = bh / (c.H >> lg), h = (bh - b * (c.H >> lg)) << lg;
  const int n_tokens = kBlockM >> lg, q_first = tile * n_tokens;
  const Rows rows{q_first, b, h, lg};
  volatile int* abort_flag = &bars.abort;

  if (warp == kWarpProducer) {
    if (lane == 0) {
      mbar_init(smem_u32(&bars.q_full), 1);
      mbar_init(smem_u32(&bars.o_full), 1);
      mbar_init(smem_u32(&bars.drain), 1);
      mbar_init(smem_u32(&bars.pv_done), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&bars.s_full[i]), 1);
        mbar_init(smem_u32(&bars.p_full[i]), 4);  // one arrive per softmax warp
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(smem_u32(&bars.k_full[i]), 1);
        mbar_init(smem_u32(&bars.k_empty[i]), 1);
        mbar_init(smem_u32(&bars.v_full[i]), 1);
        mbar_init(smem_u32(&bars.v_empty[i]), 1);
      }
      bars.abort = 0;
      fence_mbar_init();
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&bars.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_release();
  const int len = sequence_length(c, b);
  const int off = c.from_end ? len - c.Sq : c.off;
  const int last_row = min(q_first + n_tokens, c.Sq) - 1;  // a token, as q_first
  const Blocks blk = tile_blocks(c, off + q_first, off + last_row, len, rank, n_ranks);
  // The first loads go out before the block meets: nothing waits on their barriers earlier, and
  // their latency covers the rest of the set-up.
  const int kvh = c.Hkv == c.H ? h : h / (c.H / c.Hkv);
  if (warp == kWarpProducer && blk.n > 0 && lane == 0) {
    const uint32_t bar_q = smem_u32(&bars.q_full), bar_k = smem_u32(&bars.k_full[0]);
    mbar_arrive_expect_tx(bar_k, G::kTileBytes);
    mbar_arrive_expect_tx(bar_q, G::kQBytes);
#pragma unroll
    for (int bx = 0; bx < G::kBoxes; ++bx) {
      tma_load_4d(smem_base + bx * G::kQBoxBytes, &tm_q, bar_q, bx * 64, h, q_first, b);
      tma_load_4d(smem_base + G::kOffK + bx * G::kBoxBytes, &tm_k, bar_k, bx * 64, kvh, blk.base(0), b);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (warp < 4) {
    // ------------------------------------------------------------------ softmax warps
    const int row = warp * 32 + lane;
    const uint32_t lane_bits = uint32_t(warp * 32) << 16;
    const uint32_t t_s = tmem + lane_bits;
    const uint32_t t_o = tmem + lane_bits + 2 * kBlockN;
    const uint32_t bar_s0 = smem_u32(&bars.s_full[0]), bar_p0 = smem_u32(&bars.p_full[0]);
    const int q = rows.token(row);
    const bool in_range = q < c.Sq;
    const KeyRange r = visible_keys(off + min(q, c.Sq - 1), c.left, c.right, c.sinks, len);
    // keys that every row of the tile sees: blocks inside need no mask
    const KeyRange first_row = visible_keys(off + q_first, c.left, c.right, c.sinks, len);
    const KeyRange end_row = visible_keys(off + last_row, c.left, c.right, c.sinks, len);
    const int full_early = min(first_row.hi, c.sinks);
    const int full_lo = end_row.lo <= full_early ? 0 : end_row.lo, full_hi = first_row.hi;
    float m = -INFINITY;  // reference of x = s * scale * log2(e); -inf: no visible key so far
    // running sum of 2^(x - m), as two pairs of partial sums
    float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
    bool ok = true;

    for (int j = 0; j < blk.n; ++j) {
      const uint32_t buf = uint32_t(j) & 1u, round = uint32_t(j >> 1) & 1u;
      const uint32_t t_sj = t_s + buf * kBlockN;
      ok = mbar_wait(bar_s0 + 8 * buf, round, abort_flag, err, wait_limit);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      float x[kBlockN];
      {
        uint32_t t[kBlockN];
        tmem_ld64(t_sj, t);
#pragma unroll
        for (int e = 0; e < kBlockN; ++e) x[e] = __uint_as_float(t[e]);
      }
      const int kb = blk.base(j);
      if (!((kb >= full_lo && kb + kBlockN <= full_hi) || kb + kBlockN <= full_early)) {
        const int early = r.early - kb, lo = r.lo - kb, hi = r.hi - kb;  // in columns of the block
        if (__any_sync(0xffffffffu, early > 0 && early < lo)) {
          // early keys, a gap, and maybe window keys: a bit per column
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t see = (low_bits(hi - 32 * w) & ~low_bits(lo - 32 * w)) | low_bits(early - 32 * w);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see & (1u << e))) x[32 * w + e] = -INFINITY;
          }
        } else {
          // the window's ends (early keys, if any, run into it): usually one of them per block
          const int from = early >= lo ? 0 : lo;
          if (__any_sync(0xffffffffu, from > 0)) {
#pragma unroll
            for (int e = 0; e < kBlockN; ++e)
              if (e < from) x[e] = -INFINITY;
          }
          if (__any_sync(0xffffffffu, hi < kBlockN)) {
#pragma unroll
            for (int e = 0; e < kBlockN; ++e)
              if (e >= hi) x[e] = -INFINITY;
          }
        }
      }
      float mx;
      {
        float l1[22];
#pragma unroll
        for (int i = 0; i < 21; ++i) l1[i] = max3(x[3 * i], x[3 * i + 1], x[3 * i + 2]);
        l1[21] = x[63];
        float l2[8];
#pragma unroll
        for (int i = 0; i < 7; ++i) l2[i] = max3(l1[3 * i], l1[3 * i + 1], l1[3 * i + 2]);
        l2[7] = l1[21];
        mx = fmaxf(max3(l2[0], l2[1], l2[2]), max3(max3(l2[3], l2[4], l2[5]), l2[6], l2[7]));
      }
      const float m_tile = mx * scale_log2;
      float alpha = 1.0f;
      bool rescale = false;
      if (j == 0) {
        m = m_tile;
      } else {
        // a row that has seen no key yet (m = -inf) takes the block's maximum; its O is 0
        const float d = m_tile - m;
        bool grow = d > rescale_log2;
        if (!grow && d > 0.f) grow = ex2(d) * float(kMinorWeightInv - 1) >= (l0.x + l0.y) + (l1.x + l1.y);
        rescale = __any_sync(0xffffffffu, grow);
        if (rescale) {
          alpha = grow ? ex2(m - m_tile) : 1.0f;
          if (grow) m = m_tile;
          l0 = fmul2(l0, make_float2(alpha, alpha));
          l1 = fmul2(l1, make_float2(alpha, alpha));
        }
      }
      const float neg_m = m == -INFINITY ? 0.f : -m;
      const float2 sl2 = make_float2(scale_log2, scale_log2);
      const float2 nm2 = make_float2(neg_m, neg_m);
      uint32_t pk[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const float2 t = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sl2, nm2);
        const float2 pv = make_float2(ex2(t.x), ex2(t.y));  // 2^-inf = 0 for a hidden key
        if (e & 1) l1 = fadd2(l1, pv);
        else l0 = fadd2(l0, pv);
        pk[e] = pack_bf16x2(pv.x, pv.y);  // weights in bf16 for the product; l keeps fp32
      }
      tmem_st32(t_sj, pk);
      if (rescale) {
        // S ran ahead of the last block's P V, which must have left O before it is rescaled
        ok = mbar_wait(smem_u32(&bars.pv_done), uint32_t(j - 1) & 1u, abort_flag, err, wait_limit);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
        for (int oc = 0; oc < D / 32; ++oc) {
          uint32_t t[32];
          tmem_ld32(t_o + oc * 32, t);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 o = fmul2(make_float2(__uint_as_float(t[e]), __uint_as_float(t[e + 1])), a2);
            t[e] = __float_as_uint(o.x);
            t[e + 1] = __float_as_uint(o.y);
          }
          tmem_st32(t_o + oc * 32, t);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p0 + 8 * buf);
    }

    // ------------------------------------------------------------------ epilogue
    const size_t lse_idx = rows.lse(c, row);
    // Results other than a bf16 tile that leaves by TMA go through shared memory, so that a warp reads
    // 16 bytes a lane of whole rows of the running O, kBatch instructions at a time, and writes whole
    // rows.  (Each thread on its own row: 32 rows an instruction, and a read before every write.)
    constexpr bool kRun32 = kOutF32 || kResult == kMergeFrom32;
    constexpr int kCols = kRun32 ? 4 : 8, kLanes = D / kCols;  // of a lane; of a row
    constexpr int kAtOnce = 32 / kLanes, kSteps = 32 / kAtOnce, kBatch = kSteps < 16 ? kSteps : 16;
    const int sub = lane / kLanes, col = kCols * (lane % kLanes);
    // past the end any row may be read: it is not used
    const unsigned place = in_range ? rows.place(c, row) : 0u;
    const size_t out_base = rows.base(c) * D + col;
    auto row_at = [&](int s) {  // the lane's columns of the warp's row kAtOnce s + sub
      return out_base + size_t(__shfl_sync(0xffffffffu, place, kAtOnce * s + sub)) * D;
    };
    auto running = [&](int s) {
      const size_t at = row_at(s);
      if constexpr (kResult == kMergeFrom32) return *reinterpret_cast<const uint4*>(c.o_run + at);
      else if constexpr (kOutF32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(c.out) + at);
      else return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.out) + at);
    };
    uint4 run[kAcc ? kBatch : 1];
    float la = 0.f;
    if constexpr (kAcc) {
      if constexpr (!kSplit) {  // on their way while the last products run
        la = c.lse[lse_idx];
#pragma unroll
        for (int s = 0; s < kBatch; ++s) run[s] = running(s);
      }
    }
    if (ok && blk.n > 0) {
      ok = mbar_wait(smem_u32(&bars.o_full), 0, abort_flag, err, wait_limit);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc_fence_after();
      const float l = (l0.x + l0.y) + (l1.x + l1.y);
      const bool empty = l == 0.f;
      const RowEnd end = finish_row<kResult>(m, l, la, in_range);
      const float fa = end.fa, fc = kSplit ? 1.f : end.fc, lse_out = end.lse;
      const bool write = end.write;
      // O times fc into shared memory: rows of D fp32, their 16-byte vectors permuted by the row so
      // that neither writing nor reading conflicts
      const uint32_t mine = smem_base + uint32_t(warp) * 32u * D * 4u;
      auto stage = [&]() {
#pragma unroll 1
        for (int oc = 0; oc < D / 32; ++oc) {
          uint32_t t[32];
          if (blk.n > 0) tmem_ld32(t_o + oc * 32, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = empty ? 0.f : __uint_as_float(t[4 * e + i]) * fc;
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             mine + uint32_t(lane) * D * 4u + ((uint32_t(oc * 8 + e) ^ (uint32_t(lane) & 7u)) << 4)),
                         "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3])
                         : "memory");
          }
        }
      };
      if constexpr (kSplit) {  // a part, folded below
        stage();
        float* ml = reinterpret_cast<float*>(smem + G::kOffParts);
        ml[row] = m;
        ml[kBlockM + row] = l;
      } else if constexpr (!kOutF32 && !kAcc) {
        // bf16 rows go to global memory as one tile: each thread writes its row into Q's shared
        // memory (read for the last time before O was complete) in the 128-byte swizzle, and a TMA
        // store takes it from there, leaving out rows past Sq.  Row-by-row stores, 32 rows of
        // 16 bytes an instruction, kept the warps 2700 cycles and more.
        const uint32_t row_addr = smem_base + uint32_t(row) * 128u;
#pragma unroll 1
        for (int oc = 0; oc < D / 32; ++oc) {
          uint32_t t[32];
          if (blk.n > 0) tmem_ld32(t_o + oc * 32, t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = empty ? 0u : pack_bf16x2(__uint_as_float(t[8 * e + 2 * i]) * fc,
                                              __uint_as_float(t[8 * e + 2 * i + 1]) * fc);
            const uint32_t v = uint32_t((oc & 1) * 4 + e);  // 16-byte vector of the 64-column box
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             row_addr + uint32_t(oc >> 1) * G::kQBoxBytes + ((v ^ (uint32_t(row) & 7u)) << 4)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        }
        if (write && c.lse != nullptr) c.lse[lse_idx] = lse_out;
        fence_proxy_async_smem();
      } else {
        stage();
        __syncwarp();
#pragma unroll
        for (int s0 = 0; s0 < kSteps; s0 += kBatch) {
          uint4 next[kAcc ? kBatch : 1];
          if constexpr (kAcc) {
            if (s0 + kBatch < kSteps) {
#pragma unroll
              for (int s = 0; s < kBatch; ++s) next[s] = running(s0 + kBatch + s);
            }
          }
#pragma unroll
          for (int s = 0; s < kBatch; ++s) {
            const int r = kAtOnce * (s0 + s) + sub;
            float o[kCols];
#pragma unroll
            for (int v = 0; v < kCols / 4; ++v)
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(o[4 * v]), "=f"(o[4 * v + 1]), "=f"(o[4 * v + 2]), "=f"(o[4 * v + 3])
                           : "r"(mine + uint32_t(r) * D * 4u + (uint32_t(col / 4 + v) ^ (uint32_t(r) & 7u)) * 16u));
            if constexpr (kAcc) {
              const float f = __shfl_sync(0xffffffffu, fa, r);
              const uint32_t w[4] = {run[s].x, run[s].y, run[s].z, run[s].w};
              if (f != 0.f) {  // an empty running row may hold anything
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if constexpr (kRun32) {
                    o[i] = fmaf(f, __uint_as_float(w[i]), o[i]);
                  } else {
                    o[2 * i] = fmaf(f, __uint_as_float(w[i] << 16), o[2 * i]);
                    o[2 * i + 1] = fmaf(f, __uint_as_float(w[i] & 0xFFFF0000u), o[2 * i + 1]);
                  }
                }
              }
            }
            const int live = __shfl_sync(0xffffffffu, int(write), r);
            const size_t at = row_at(s0 + s);
            if (live) {
              if constexpr (kOutF32)
                *reinterpret_cast<float4*>(static_cast<float*>(c.out) + at) = make_float4(o[0], o[1], o[2], o[3]);
              else if constexpr (kCols == 4)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.out) + at) =
                    make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
              else
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out) + at) =
                    make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                               pack_bf16x2(o[6], o[7]));
            }
          }
          if constexpr (kAcc) {
#pragma unroll
            for (int s = 0; s < kBatch; ++s) run[s] = next[s];
          }
        }
        if (write && c.lse != nullptr) c.lse[lse_idx] = lse_out;
      }
    }
    if constexpr (!kOutF32 && !kAcc) {
      // every softmax warp comes here, also one whose wait ran out
      if (!kSplit && bar_and(1, 128, ok) && threadIdx.x == 0) {
#pragma unroll
        for (int bx = 0; bx < G::kBoxes; ++bx)
          tma_store_4d(&tm_o, smem_base + bx * G::kQBoxBytes, bx * 64, h, q_first, b);
        tma_store_wait();
      }
    }
  } else if (warp == kWarpProducer) {
    // ------------------------------------------------------------------ TMA producer
    if (blk.n > 0 && lane == 0) {
      const uint32_t bar_q = smem_u32(&bars.q_full);
      int k_issued = 1, v_issued = 0;  // K of block 0 and Q are on their way
      for (int j = 0; j < blk.n; ++j) {
        const int kb = blk.base(j);
        const int ks = j % G::kK;
        if (j > 0) {
          if (!mbar_wait(smem_u32(&bars.k_empty[ks]), (uint32_t(j / G::kK) & 1u) ^ 1u, abort_flag, err,
                         wait_limit))
            break;
          const uint32_t bar_k = smem_u32(&bars.k_full[ks]);
          mbar_arrive_expect_tx(bar_k, G::kTileBytes);
#pragma unroll
          for (int bx = 0; bx < G::kBoxes; ++bx)
            tma_load_4d(smem_base + G::kOffK + ks * G::kTileBytes + bx * G::kBoxBytes, &tm_k, bar_k, bx * 64,
                        kvh, kb, b);
          k_issued = j + 1;
        }
        const int vs = j % G::kV;
        if (!mbar_wait(smem_u32(&bars.v_empty[vs]), (uint32_t(j / G::kV) & 1u) ^ 1u, abort_flag, err, wait_limit))
          break;
        const uint32_t bar_v = smem_u32(&bars.v_full[vs]);
        mbar_arrive_expect_tx(bar_v, G::kTileBytes);
#pragma unroll
        for (int bx = 0; bx < G::kBoxes; ++bx)
          tma_load_4d(smem_base + G::kOffV + vs * G::kTileBytes + bx * G::kBoxBytes, &tm_v, bar_v, bx * 64, kvh, kb, b);
        v_issued = j + 1;
      }
      // every issued copy lands before the CTA's shared memory is released
      drain_wait(bar_q, 0, wait_limit);
      for (int j = k_issued > G::kK ? k_issued - G::kK : 0; j < k_issued; ++j)
        drain_wait(smem_u32(&bars.k_full[j % G::kK]), uint32_t(j / G::kK) & 1u, wait_limit);
      for (int u = v_issued > G::kV ? v_issued - G::kV : 0; u < v_issued; ++u)
        drain_wait(smem_u32(&bars.v_full[u % G::kV]), uint32_t(u / G::kV) & 1u, wait_limit);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA issuer
    // one thread issues; the whole warp only meets to clear hidden V rows
    if (blk.n > 0) {
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, D, true);
      const uint64_t q_desc = sdesc_sw128(smem_base, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_base + G::kOffK, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_base + G::kOffV, G::kBoxBytes, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait(smem_u32(bar), parity & 1u, abort_flag, err, wait_limit);
      };
      // S = Q K^T of block j into buffer j & 1, over D in K = 16 steps: 32 bytes per step inside a
      // 128-byte swizzled row, the next 64 columns in the next box
      auto issue_qk = [&](int j) {
        const int ks = j % G::kK;
        if (!wait(&bars.k_full[ks], uint32_t(j / G::kK))) return false;
        tc_fence_after();
        const uint64_t kd = k_desc + uint32_t(ks * (G::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t qo = ((kk >> 2) * G::kQBoxBytes + (kk & 3) * 32) >> 4;
          const uint32_t ko = ((kk >> 2) * G::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss(tmem + (j & 1) * kBlockN, q_desc + qo, kd + ko, idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars.s_full[j & 1]));
        tc_commit(smem_u32(&bars.k_empty[ks]));
        return true;
      };
      bool ok = true;
      if (leader) {
        ok = wait(&bars.q_full, 0) && issue_qk(0);
        if (blk.n > 1) ok = ok && issue_qk(1);
      }
      int vs = 0;
      uint32_t v_round = 0;
      for (int j = 0; j < blk.n; ++j) {
        const int kb = blk.base(j);
        const int k1 = min(kb + kBlockN, c.Skv);  // rows past Skv arrive as 0
        if (!blk.all_seen(kb, k1)) {
          bool landed = wait(&bars.v_full[vs], v_round);
          landed = __all_sync(0xffffffffu, landed);
          // the hidden rows are [early, lo) and [hi, ..) of the block: whole 128-byte rows of each
          // box, whatever the swizzle, so runs of 16-byte stores
          uint8_t* v = smem + G::kOffV + vs * G::kTileBytes;
          auto clear = [&](int r0, int r1) {
            for (int o = r0 * 128 + lane * 16; o < r1 * 128; o += 512)
#pragma unroll
              for (int bx = 0; bx < G::kBoxes; ++bx)
                *reinterpret_cast<uint4*>(v + bx * G::kBoxBytes + o) = make_uint4(0u, 0u, 0u, 0u);
          };
          if (landed) {
            clear(max(blk.early - kb, 0), min(blk.lo, k1) - kb);
            clear(max(blk.hi - kb, 0), k1 - kb);
          }
          fence_proxy_async_smem();  // the tensor core reads the zeros
          __syncwarp();
        }
        if (leader && ok) {
          ok = wait(&bars.v_full[vs], v_round) && wait(&bars.p_full[j & 1], uint32_t(j >> 1));
          if (ok) {
            tc_fence_after();
            // O += P V over the 64 keys in K = 16 steps: P from TMEM (8 columns per step), V MN-major
            // (16 key rows = 2 KB per step, the next 64 columns of D in the next box)
            const uint64_t vd = v_desc + uint32_t(vs * (G::kTileBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < kBlockN / 16; ++kk)
              mma_ts(tmem + 2 * kBlockN, tmem + (j & 1) * kBlockN + kk * 8, vd + uint32_t((kk * 16 * 128) >> 4), idesc_pv,
                     (j > 0 || kk > 0) ? 1u : 0u);
            tc_commit(smem_u32(&bars.v_empty[vs]));
            tc_commit(smem_u32(&bars.pv_done));
            if (j + 2 < blk.n) ok = issue_qk(j + 2);  // over P of this block, after its product
          }
        }
        __syncwarp();
        if (++vs == G::kV) {
          vs = 0;
          ++v_round;
        }
      }
      if (leader) {
        if (ok) tc_commit(smem_u32(&bars.o_full));
        tc_commit(smem_u32(&bars.drain));  // no MMA may still be writing TMEM when it is freed
        drain_wait(smem_u32(&bars.drain), 0, wait_limit);
      }
      __syncwarp();
    }
  }

  if constexpr (kSplit) {
    // fold the parts: each block finishes 128 / n_ranks rows, the sums in the order of the parts
    cluster.sync();
    if (warp < 4) {
      if (n_ranks == 2) fold_parts<D, kOutF32, kResult, 2>(c, cluster, smem, rows);
      else if (n_ranks == 4) fold_parts<D, kOutF32, kResult, 4>(c, cluster, smem, rows);
      else fold_parts<D, kOutF32, kResult, 8>(c, cluster, smem, rows);
    }
    cluster.sync();  // no block leaves while another reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

// [B][S][H][D] bf16 tensor whose tokens are `stride` elements apart: 64 columns x `heads` heads x
// `tokens` tokens x 1 batch, 128-byte swizzle; tokens past S read as 0.
bool encode(CUtensorMap* map, const void* ptr, int B, int S, int H, int D, long long stride, unsigned tokens,
            unsigned heads) {
  auto fn = tensor_map_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(S), cuuint64_t(B)};
  const cuuint64_t token = cuuint64_t(stride) * 2;
  const cuuint64_t strides[3] = {cuuint64_t(D) * 2, token, B > 1 ? token * cuuint64_t(S) : token};
  const cuuint32_t box[4] = {64, heads, tokens, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Heads of a key head that a tile takes together, as a power of two.  Tokens then span fewer keys and
// few of them still fill a tile: 16000 x 32 heads on 8, causal window 2000, 579 -> 530 us, 4000 x 32 on
// 8, window 100, 40 -> 34.5; 16 tokens of 8 sequences x 32 heads on 8 against 4096 keys 77 -> 35.
int heads_log2(const WindowCall& c) {
  int lg = 0;
  while (lg < 7 && (c.H / c.Hkv) % (2 << lg) == 0) ++lg;
  return lg;
}

long long tiles(const WindowCall& c, int lg) {
  const int n = kBlockM >> lg;
  return ((long long)c.Sq + n - 1) / n * (c.H >> lg) * c.B;
}

// Blocks that share a query tile's keys, and the time (us) that the kernel is then expected to take.  A
// tile walks 0.66 us per block of 64 keys, 0.95 beside another on its SM; parts cost 1.9 us to
// start and fold, 4 when they are more than the SMs.  Clusters of four and eight do not fill
// every SM.  Measured, parts 1 / 2 / 4 / 8: 20 tiles of 512 keys 9.9 / 9.2 / 7.9 / 10.3 us, of 2048
// 25.8 / 17.5 / 12.6 / 14.1; 100 tiles of 1024 15.7 / 16.2 (200 blocks), of 4096 47.6 / 38.2; 48 tiles of
// 2048 26.5 / 18.5 / 18.1; 37 tiles of 512 10.1 / 9.4 / 10.7 / 16.9.
struct Plan {
  int parts;
  double us;
};

Plan plan(const WindowCall& c) {
  const int lg = heads_log2(c);
  const long long items = tiles(c, lg), sms = sm_count(), span = kBlockM >> lg;
  long long keys = c.Skv, early = 0;  // of a tile, at most
  if (c.left >= 0 && c.right >= 0 && c.left + c.right + span < keys) {
    keys = c.left + c.right + span;
    early = c.sinks < c.Skv - keys ? c.sinks : c.Skv - keys;
  }
  const long long blocks = (keys + kBlockN - 1) / kBlockN + (early + kBlockN - 1) / kBlockN;
  if (items > sms) return {1, 5.0 + double((items + 2 * sms - 1) / (2 * sms)) * double(blocks) * 1.2};
  Plan best{1, 5.0 + 0.66 * double(blocks)};
  for (int n = 2; n <= kMaxCluster && 2 * items * n <= (n == 2 ? 4 : 3) * sms; n *= 2) {
    const double own = double((blocks + n - 1) / n);
    const double t = 5.0 + (items * n * (n == 2 ? 20 : 23) <= 20 * sms ? 1.9 + 0.66 * own : 4.0 + 0.95 * own);
    if (t < best.us) best = {n, t};
  }
  return best;
}

template <int D, bool kOutF32, int kResult, bool kSplit>
cudaError_t launch_parts(const WindowCall& c, int n_ranks, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& to, int* err, cudaStream_t stream) {
  auto kernel = window_sm100_kernel<D, kOutF32, kResult, kSplit>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(reinterpret_cast<const void*>(kernel), Geometry<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int lg = heads_log2(c);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles(c, lg) * n_ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Geometry<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(n_ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, c, to, lg,
                            float(double(c.scale) * 1.4426950408889634074),
                            kRescaleLog2, err, kDefaultWaitLimit);
}

template <int D, bool kOutF32, int kResult>
cudaError_t launch(const WindowCall& c, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& to, int* err, cudaStream_t stream) {
  const int n = plan(c).parts;
  return n > 1 ? launch_parts<D, kOutF32, kResult, true>(c, n, tq, tk, tv, to, err, stream)
               : launch_parts<D, kOutF32, kResult, false>(c, 1, tq, tk, tv, to, err, stream);
}

template <int D>
cudaError_t launch_d(const WindowCall& c, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& to, int* err, cudaStream_t stream) {
  if (c.out_f32)
    return c.accumulate ? launch<D, true, kMerge>(c, tq, tk, tv, to, err, stream)
                        : launch<D, true, kWrite>(c, tq, tk, tv, to, err, stream);
  if (!c.accumulate) return launch<D, false, kWrite>(c, tq, tk, tv, to, err, stream);
  return c.o_run != nullptr ? launch<D, false, kMergeFrom32>(c, tq, tk, tv, to, err, stream)
                            : launch<D, false, kMerge>(c, tq, tk, tv, to, err, stream);
}

}  // namespace

double window_sm100_us(const WindowCall& c) { return plan(c).us; }

cudaError_t launch_window_sm100(const WindowCall& c, int* err, cudaStream_t stream) {
  const int lg = heads_log2(c);
  CUtensorMap tq, tk, tv, to;
  if (!encode(&tq, c.q, c.B, c.Sq, c.H, c.D, c.q_stride, kBlockM >> lg, 1u << lg)) return cudaErrorInvalidValue;
  if (c.Skv == 0) tk = tv = tq;  // no block loads through them
  else if (!encode(&tk, c.k, c.B, c.Skv, c.Hkv, c.D, c.k_stride, kBlockN, 1) ||
           !encode(&tv, c.v, c.B, c.Skv, c.Hkv, c.D, c.v_stride, kBlockN, 1))
    return cudaErrorInvalidValue;
  // bf16 results leave by TMA; the other forms do not use the map
  if (c.out_f32 || c.accumulate) to = tq;
  else if (!encode(&to, c.out, c.B, c.Sq, c.H, c.D, (long long)c.H * c.D, kBlockM >> lg, 1u << lg))
    return cudaErrorInvalidValue;
  return c.D == 128 ? launch_d<128>(c, tq, tk, tv, to, err, stream) : launch_d<64>(c, tq, tk, tv, to, err, stream);
}

}  // namespace cpattn
