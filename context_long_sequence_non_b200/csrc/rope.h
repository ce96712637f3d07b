// rope.h -- internal launchers of the rotary-position kernels (rope_api.cu checks every
// argument before any of them runs).
#pragma once

#include <cuda_runtime.h>

namespace cpattn {

constexpr int kRopeMaxD = 256;

// One tensor of a call: token t's head h is read at src + t * src_stride + h * D and written at
// dst + (h / group) * group_stride + t * dst_stride + (h % group) * D  (elements).
struct RopeTensor {
  const void* src;
  void* dst;
  const float* gamma;  // RMSNorm weights; nullptr: not normalised
  long long src_stride, dst_stride, group_stride;
  int heads, group;
  bool rotate;
  unsigned group_magic;  // filled in by the launcher
};

// Up to three tensors of the same tokens.  The angle of pair p at token t is
//   sum_a pos[t % pos_rows][a] * freq[a][p]   (a < n_axes, p < rot / 2).
struct RopeCall {
  RopeTensor t[3];
  int n_tensors;
  const int* pos;
  const double* freq;
  int tokens, pos_rows, D, rot, n_axes;
  bool interleaved, f32;
  float factor, eps, out_scale;
};

cudaError_t launch_rope(const RopeCall& c, cudaStream_t stream);

}  // namespace cpattn
