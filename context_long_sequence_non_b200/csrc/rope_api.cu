// rope_api.cu -- the C entry points of the rotary positions and of the Q/K norm with rotation:
// argument checks (all before the first CUDA call), the frequency rules, and dispatch.
#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "cpattn.h"
#include "kernels.h"
#include "rope.h"

using cpattn::aligned;
using cpattn::cuda_status;
using cpattn::elem_size;
using cpattn::overlap;
using cpattn::RopeCall;
using cpattn::RopeTensor;

namespace {

// Do two sets of evenly spaced token rows (in bytes) share a byte?  Exact when the spacings
// agree -- the interleaved heads of one projection's output do not overlap -- and the plain
// test of their extents otherwise.
bool rows_overlap(const void* a, size_t row_a, size_t step_a, const void* b, size_t row_b,
                  size_t step_b, size_t tokens) {
  const size_t na = (tokens - 1) * step_a + row_a, nb = (tokens - 1) * step_b + row_b;
  if (!overlap(a, na, b, nb)) return false;
  if (step_a != step_b || tokens == 1) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t d = y >= x ? (y - x) % step_a : (step_a - (x - y) % step_a) % step_a;  // b after a
  return d < row_a || step_a - d < row_b;
}

// Checks shared by the three calls.  Every tensor's rows must be packed heads; `scattered`
// (the re-partition) writes one contiguous block of tokens x heads x D elements instead.
int check(RopeCall* c, int dtype, bool scattered) {
  if (c->tokens < 0 || c->D < 2 || c->D > cpattn::kRopeMaxD) return CPATTN_ERR_SHAPE;
  if (c->rot < 2 || c->rot > c->D || c->rot % 2 != 0) return CPATTN_ERR_SHAPE;
  if (c->n_axes < 1 || c->n_axes > 4) return CPATTN_ERR_SHAPE;
  if (!std::isfinite(c->factor) || !std::isfinite(c->out_scale) || !std::isfinite(c->eps) || c->eps < 0.f)
    return CPATTN_ERR_SHAPE;
  const int es = elem_size(dtype);
  if (es == 0) return CPATTN_ERR_UNSUPPORTED;
  c->f32 = dtype == CPATTN_F32;
  long long heads = 0;
  for (int i = 0; i < c->n_tensors; ++i) {
    RopeTensor& t = c->t[i];
    if (t.heads < 1 || t.heads > 65535) return CPATTN_ERR_SHAPE;
    heads += t.heads;
    const long long row = (long long)t.heads * c->D;
    if (t.src_stride == 0) t.src_stride = row;
    if (t.dst_stride == 0) t.dst_stride = row;
    if (t.src_stride < row || (!scattered && t.dst_stride < row)) return CPATTN_ERR_SHAPE;
    // 2^31 tokens less than 2^30 elements apart: every extent below fits 64 bits
    if (t.src_stride >= (1LL << 30) || t.dst_stride >= (1LL << 30)) return CPATTN_ERR_SHAPE;
  }
  if (c->tokens == 0) return CPATTN_OK;  // nothing is read or written: pointers are not checked
  if (c->pos_rows < 1 || c->tokens % c->pos_rows != 0) return CPATTN_ERR_SHAPE;
  if ((long long)c->tokens * heads > 0x7fffffffLL - 4096) return CPATTN_ERR_SHAPE;  // 32-bit rows
  if (c->pos == nullptr || c->freq == nullptr) return CPATTN_ERR_NULL;
  for (int i = 0; i < c->n_tensors; ++i)
    if (c->t[i].src == nullptr || c->t[i].dst == nullptr) return CPATTN_ERR_NULL;
  if (!aligned(c->pos, 4) || !aligned(c->freq, 8)) return CPATTN_ERR_ALIGN;
  const size_t n = size_t(c->tokens);
  for (int i = 0; i < c->n_tensors; ++i) {
    const RopeTensor& d = c->t[i];
    if (!aligned(d.src, 16) || !aligned(d.dst, 16) || (d.gamma != nullptr && !aligned(d.gamma, 16)))
      return CPATTN_ERR_ALIGN;
    const size_t d_row = scattered ? n * d.heads * c->D * es : size_t(d.heads) * c->D * es;
    const size_t d_step = scattered ? d_row : size_t(d.dst_stride) * es;
    const size_t d_n = scattered ? 1 : n;
    const size_t d_span = (d_n - 1) * d_step + d_row;
    for (int j = 0; j < c->n_tensors; ++j) {
      const RopeTensor& s = c->t[j];
      const size_t s_row = size_t(s.heads) * c->D * es, s_step = size_t(s.src_stride) * es;
      const bool same = i == j && !scattered && d.src == d.dst && s_step == d_step;  // in place
      const bool clash = scattered
          ? overlap(d.dst, d_span, s.src, (n - 1) * s_step + s_row)
          : rows_overlap(d.dst, d_row, d_step, s.src, s_row, s_step, n);
      if (!same && clash) return CPATTN_ERR_SHAPE;
      const size_t e_row = scattered ? n * s.heads * c->D * es : s_row;
      const size_t e_step = scattered ? e_row : size_t(s.dst_stride) * es;
      if (i != j && rows_overlap(d.dst, d_row, d_step, s.dst, e_row, e_step, d_n)) return CPATTN_ERR_SHAPE;
      if (s.gamma != nullptr && overlap(d.dst, d_span, s.gamma, size_t(c->D) * 4)) return CPATTN_ERR_SHAPE;
    }
    if (overlap(d.dst, d_span, c->pos, size_t(c->pos_rows) * c->n_axes * 4) ||
        overlap(d.dst, d_span, c->freq, size_t(c->n_axes) * (c->rot / 2) * 8))
      return CPATTN_ERR_SHAPE;
  }
  return CPATTN_OK;
}

int launch(const RopeCall& c, cpattn_stream_t stream) {
  if (c.tokens == 0) return CPATTN_OK;
  return cuda_status(cpattn::launch_rope(c, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int cpattn_rope_frequencies(double* freq, float* factor, int rot, double base, int scaling,
                            double stretch, double train_len, double beta_fast, double beta_slow) {
  constexpr double kTwoPi = 6.28318530717958647693;
  if (rot < 2 || rot % 2 != 0 || rot > cpattn::kRopeMaxD) return CPATTN_ERR_SHAPE;
  if (!(std::isfinite(base) && base > 1.0)) return CPATTN_ERR_SHAPE;
  if (scaling < CPATTN_ROPE_PLAIN || scaling > CPATTN_ROPE_BY_PARTS) return CPATTN_ERR_UNSUPPORTED;
  if (scaling != CPATTN_ROPE_PLAIN && !(std::isfinite(stretch) && stretch >= 1.0)) return CPATTN_ERR_SHAPE;
  if (scaling == CPATTN_ROPE_NTK && rot < 4) return CPATTN_ERR_SHAPE;
  if (scaling == CPATTN_ROPE_BY_PARTS &&
      !(std::isfinite(train_len) && train_len > 0.0 && std::isfinite(beta_fast) && std::isfinite(beta_slow) &&
        beta_slow > 0.0 && beta_fast > beta_slow))
    return CPATTN_ERR_SHAPE;
  if (freq == nullptr) return CPATTN_ERR_NULL;
  if (scaling == CPATTN_ROPE_NTK) base *= std::pow(stretch, double(rot) / (rot - 2));
  for (int p = 0; p < rot / 2; ++p) {
    double w = std::pow(base, -2.0 * p / rot);
    if (scaling == CPATTN_ROPE_LINEAR) w /= stretch;
    if (scaling == CPATTN_ROPE_BY_PARTS) {
      const double turns = train_len * w / kTwoPi;  // full turns over the trained length
      double keep = (turns - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      w = w / stretch * (1.0 - keep) + w * keep;
    }
    freq[p] = w;
  }
  if (factor != nullptr)
    *factor = scaling == CPATTN_ROPE_BY_PARTS ? float(0.1 * std::log(stretch) + 1.0) : 1.0f;
  return CPATTN_OK;
}

int cpattn_rope(const void* x, void* y, const int* pos, const double* freq, int tokens, int pos_rows,
                int H, int D, int rot, int n_axes, int interleaved, float factor, long long x_stride,
                long long y_stride, int dtype, cpattn_stream_t stream) {
  RopeCall c{};
  c.n_tensors = 1;
  c.t[0] = RopeTensor{x, y, nullptr, x_stride, y_stride, 0, H, H, true, 0};
  c.pos = pos, c.freq = freq, c.tokens = tokens, c.pos_rows = pos_rows, c.D = D, c.rot = rot;
  c.n_axes = n_axes, c.interleaved = interleaved != 0, c.factor = factor, c.eps = 0.f, c.out_scale = 1.f;
  const int st = check(&c, dtype, false);
  return st != CPATTN_OK ? st : launch(c, stream);
}

int cpattn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const float* gamma_q,
                        const float* gamma_k, const int* pos, const double* freq, int tokens,
                        int pos_rows, int Hq, int Hk, int D, int rot, int n_axes, int interleaved,
                        float eps, float out_scale, float factor, long long q_stride,
                        long long k_stride, long long q_out_stride, long long k_out_stride, int dtype,
                        cpattn_stream_t stream) {
  RopeCall c{};
  c.n_tensors = 2;
  c.t[0] = RopeTensor{q, q_out, gamma_q, q_stride, q_out_stride, 0, Hq, Hq, true, 0};
  c.t[1] = RopeTensor{k, k_out, gamma_k, k_stride, k_out_stride, 0, Hk, Hk, true, 0};
  c.pos = pos, c.freq = freq, c.tokens = tokens, c.pos_rows = pos_rows, c.D = D, c.rot = rot;
  c.n_axes = n_axes, c.interleaved = interleaved != 0, c.factor = factor, c.eps = eps, c.out_scale = out_scale;
  const int st = check(&c, dtype, false);
  if (st != CPATTN_OK) return st;
  if (tokens > 0 && (gamma_q == nullptr || gamma_k == nullptr)) return CPATTN_ERR_NULL;
  return launch(c, stream);
}

int cpattn_seq2head_qkv_norm_rope(const void* q, const void* k, const void* v, void* qh, void* kh,
                                  void* vh, const float* gamma_q, const float* gamma_k, const int* pos,
                                  const double* freq, int P, int S_local, int H, int D, int rot,
                                  int n_axes, int interleaved, float eps, float out_scale, float factor,
                                  cpattn_stream_t stream) {
  if (P < 1 || S_local < 1 || H < 1 || D < 2 || H % P != 0) return CPATTN_ERR_SHAPE;
  if ((long long)P * S_local > 0x7fffffffLL) return CPATTN_ERR_SHAPE;
  if ((long long)(H / P) * D * 2 % 16 != 0) return CPATTN_ERR_SHAPE;  // as cpattn_seq2head
  if ((gamma_q == nullptr) != (gamma_k == nullptr)) return CPATTN_ERR_NULL;
  const int Hp = H / P, T = P * S_local;
  const long long group = (long long)T * Hp * D, row = (long long)Hp * D;
  RopeCall c{};
  c.n_tensors = 3;
  c.t[0] = RopeTensor{q, qh, gamma_q, 0, row, group, H, Hp, true, 0};
  c.t[1] = RopeTensor{k, kh, gamma_k, 0, row, group, H, Hp, true, 0};
  c.t[2] = RopeTensor{v, vh, nullptr, 0, row, group, H, Hp, false, 0};
  c.pos = pos, c.freq = freq, c.tokens = T, c.pos_rows = T, c.D = D, c.rot = rot;
  c.n_axes = n_axes, c.interleaved = interleaved != 0, c.factor = factor, c.eps = eps, c.out_scale = out_scale;
  const int st = check(&c, CPATTN_BF16, true);
  return st != CPATTN_OK ? st : launch(c, stream);
}

}  // extern "C"
