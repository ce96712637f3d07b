// window.h -- internal launchers of the windowed attention (window_api.cu checks every
// argument before any of them runs).
#pragma once

#include <cuda_runtime.h>

namespace cpattn {

// One windowed attention call.  Positions are relative to key row 0: query row i sits at
// off + i, key row j at j.  Key j is visible to query position p when
//   j < len  and  (right < 0 or j <= p + right)  and  (left < 0 or j >= p - left or j < sinks)
// with len = Skv, or clamp(kv_len[b], 0, Skv) when kv_len is given.  from_end: the queries are
// the last Sq tokens of each sequence, off = len - Sq.
struct WindowCall {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int* kv_len;
  const float* o_run;  // accumulate: the running O, when it is not `out` itself
  int B, H, Hkv, Sq, Skv, D;
  long long q_stride, k_stride, v_stride;  // elements between tokens; a batch is S tokens
  float scale;
  int off, left, right, sinks;
  bool from_end, in_f32, out_f32, accumulate;
};

// A query position's visible keys as two ranges: [0, early) and [lo, hi), early <= lo <= hi.
struct KeyRange {
  int early, lo, hi;
};

__host__ __device__ inline KeyRange visible_keys(int p, int left, int right, int sinks, int len) {
  KeyRange r;
  r.hi = len;
  if (right >= 0 && p + right + 1 < len) r.hi = p + right + 1;
  if (r.hi < 0) r.hi = 0;
  r.lo = left < 0 || p < left ? 0 : p - left;
  if (r.lo > r.hi) r.lo = r.hi;
  r.early = sinks < r.lo ? sinks : r.lo;
  return r;
}

__device__ __forceinline__ int sequence_length(const WindowCall& c, int b) {
  if (c.kv_len == nullptr) return c.Skv;
  const int n = c.kv_len[b];
  return n < 0 ? 0 : (n > c.Skv ? c.Skv : n);
}

// fp32 inputs, D <= 256, both forms (no accumulate).
cudaError_t launch_window_f32(const WindowCall& c, cudaStream_t stream);

// Tensor-core kernel: bf16 inputs, D 64 or 128; and the time in microseconds to expect of it.
cudaError_t launch_window_sm100(const WindowCall& c, int* err, cudaStream_t stream);
double window_sm100_us(const WindowCall& c);

// Single-token form (from_end, right = 0): bf16 inputs, D 64 or 128.
cudaError_t launch_window_decode(const WindowCall& c, cudaStream_t stream);

}  // namespace cpattn
