// window_api.cu -- the C entry points of windowed attention and its single-token form:
// argument checks (all before the first CUDA call) and dispatch.
#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "cpattn.h"
#include "kernels.h"
#include "window.h"

using cpattn::aligned;
using cpattn::cuda_status;
using cpattn::elem_size;
using cpattn::overlap;
using cpattn::WindowCall;

namespace {

constexpr int kMaxPos = 1 << 30;  // positions stay below this, so position arithmetic fits an int

int clamp_extent(int n) { return n < 0 ? -1 : (n >= kMaxPos ? kMaxPos - 1 : n); }

// Bytes from the first to the last element of n tokens of `row` elements each, `stride` apart (at
// most 2^30 tokens a batch, less than 2^40 bytes apart: capped where that passes any memory).
size_t span_bytes(long long tokens, long long stride, long long row, int es) {
  if (tokens < 1) return 0;
  const double bytes = (double(tokens - 1) * double(stride) + double(row)) * es;
  return bytes > 1e18 ? size_t(1) << 60 : size_t((tokens - 1) * stride + row) * es;
}

// Checks shared by both calls; fills the strides in (0: packed).
int check(WindowCall* c, int in_dtype, int out_dtype) {
  if (c->B < 1 || c->H < 1 || c->Hkv < 1 || c->Sq < 1 || c->Skv < 0 || c->D < 1) return CPATTN_ERR_SHAPE;
  if (c->H % c->Hkv != 0 || c->B > 65535 || c->H > 65535) return CPATTN_ERR_SHAPE;
  if (c->Sq >= kMaxPos || c->Skv >= kMaxPos) return CPATTN_ERR_SHAPE;
  if ((long long)c->B * c->Sq * c->H > 0x7fffffffLL) return CPATTN_ERR_SHAPE;  // 32-bit row index
  if (!(std::isfinite(c->scale) && c->scale > 0.f) || c->sinks < 0) return CPATTN_ERR_SHAPE;
  const int es = elem_size(in_dtype), oes = elem_size(out_dtype);
  if (es == 0 || oes == 0) return CPATTN_ERR_UNSUPPORTED;
  if (in_dtype == CPATTN_BF16 && c->D != 64 && c->D != 128) return CPATTN_ERR_UNSUPPORTED;
  if (in_dtype == CPATTN_F32 && c->D > 256) return CPATTN_ERR_UNSUPPORTED;
  if (c->accumulate && in_dtype != CPATTN_BF16) return CPATTN_ERR_UNSUPPORTED;
  const long long q_row = (long long)c->H * c->D, kv_row = (long long)c->Hkv * c->D;
  if (c->q_stride == 0) c->q_stride = q_row;
  if (c->k_stride == 0) c->k_stride = kv_row;
  if (c->v_stride == 0) c->v_stride = kv_row;
  if (c->q_stride < q_row || c->k_stride < kv_row || c->v_stride < kv_row) return CPATTN_ERR_SHAPE;
  // a tensor map's strides are below 2^40 bytes, from token to token and from batch to batch
  const int q_steps = c->B > 1 ? c->Sq : 1, kv_steps = c->B > 1 && c->Skv > 1 ? c->Skv : 1;
  const long long most = (1LL << 40) / es - 1;
  if (c->q_stride > most / q_steps || c->k_stride > most / kv_steps || c->v_stride > most / kv_steps)
    return CPATTN_ERR_SHAPE;
  if (c->q == nullptr || c->out == nullptr || (c->accumulate && c->lse == nullptr)) return CPATTN_ERR_NULL;
  if (c->Skv > 0 && (c->k == nullptr || c->v == nullptr)) return CPATTN_ERR_NULL;
  if (!aligned(c->q, 16) || !aligned(c->out, 16) || (c->lse != nullptr && !aligned(c->lse, 4)) ||
      (c->kv_len != nullptr && !aligned(c->kv_len, 4)) ||
      (c->Skv > 0 && (!aligned(c->k, 16) || !aligned(c->v, 16))))
    return CPATTN_ERR_ALIGN;
  if (in_dtype == CPATTN_BF16 && (c->q_stride % 8 || c->k_stride % 8 || c->v_stride % 8))
    return CPATTN_ERR_ALIGN;  // 16-byte token rows
  // the outputs are written while the inputs are still read
  const size_t ob = size_t(c->B) * c->Sq * c->H * c->D * oes, lb = size_t(c->B) * c->H * c->Sq * 4;
  const size_t qb = span_bytes((long long)c->B * c->Sq, c->q_stride, q_row, es);
  const size_t kb = span_bytes((long long)c->B * c->Skv, c->k_stride, kv_row, es);
  const size_t vb = span_bytes((long long)c->B * c->Skv, c->v_stride, kv_row, es);
  const void* in[3] = {c->q, c->k, c->v};
  const size_t in_b[3] = {qb, kb, vb};
  for (int t = 0; t < 3; ++t)
    if (in_b[t] > 0 && (overlap(c->out, ob, in[t], in_b[t]) ||
                        (c->lse != nullptr && overlap(c->lse, lb, in[t], in_b[t]))))
      return CPATTN_ERR_SHAPE;
  if (c->lse != nullptr && overlap(c->out, ob, c->lse, lb)) return CPATTN_ERR_SHAPE;
  if (c->kv_len != nullptr && (overlap(c->out, ob, c->kv_len, size_t(c->B) * 4) ||
                               (c->lse != nullptr && overlap(c->lse, lb, c->kv_len, size_t(c->B) * 4))))
    return CPATTN_ERR_SHAPE;
  c->in_f32 = in_dtype == CPATTN_F32;
  c->out_f32 = out_dtype == CPATTN_F32;
  return CPATTN_OK;
}

// Which kernel serves `window_decode`: the split one, which reads a sequence's keys once for every 16
// (token, head) rows, or, for many tokens and heads, the tensor-core one with its 128-row tiles.
// The split kernel's passes of 4 D bytes a key come out of L2 at 7.8 TB/s; the other knows its time.
// Measured, split / tiles (us): 8 sequences x 32 heads on 8, D = 128, a window of 4096, 38 / 34 at 8
// tokens, 138 / 36 at 32; 64 x 128 heads on 16, 5 tokens, 4000 keys, 533 / 279; 1 x 16 heads on 16,
// 16 / 17 at 32 tokens, 22 / 18 at 64; 32 x 16 heads on 2, 2 tokens, 1000 keys, 10 / 13.
bool tiles_serve(const WindowCall& c) {
  const double passes = double(c.B) * c.Hkv * (((long long)(c.H / c.Hkv) * c.Sq + 15) / 16);
  double keys = c.Skv;
  if (c.left >= 0 && double(c.sinks) + c.left + c.Sq < keys) keys = double(c.sinks) + c.left + c.Sq;
  return cpattn::window_sm100_us(c) < 3.5 + passes * keys * 4 * c.D / 7.8e6;
}

}  // namespace

extern "C" {

int cpattn_window_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
                      const int* kv_len, const float* o_run, int B, int H, int Hkv, int Sq, int Skv, int D,
                      long long q_stride, long long k_stride, long long v_stride, float scale,
                      int q_pos, int k_pos, int left, int right, int sinks, int in_dtype,
                      int out_dtype, int accumulate, cpattn_stream_t stream) {
  WindowCall c{q, k, v, out, lse, kv_len, o_run, B, H, Hkv, Sq, Skv, D, q_stride, k_stride, v_stride, scale,
               0, clamp_extent(left), clamp_extent(right), sinks, false, false, false, accumulate != 0};
  const int st = check(&c, in_dtype, out_dtype);
  if (st != CPATTN_OK) return st;
  if (o_run != nullptr) {
    if (accumulate == 0 || out_dtype != CPATTN_BF16) return CPATTN_ERR_UNSUPPORTED;
    if (!aligned(o_run, 16)) return CPATTN_ERR_ALIGN;
    const size_t n = size_t(B) * Sq * H * D, lb = size_t(B) * H * Sq * 4;
    if (overlap(o_run, n * 4, out, n * 2) || overlap(o_run, n * 4, lse, lb)) return CPATTN_ERR_SHAPE;
  }
  if (q_pos < 0 || k_pos < 0 || q_pos >= kMaxPos - Sq || k_pos >= kMaxPos - Skv) return CPATTN_ERR_SHAPE;
  c.off = q_pos - k_pos;
  c.sinks = sinks <= k_pos ? 0 : (sinks - k_pos < Skv ? sinks - k_pos : Skv);
  // a chunk that no row can see adds nothing to a running result
  const int last = c.off + Sq - 1;
  const bool none = Skv == 0 || (c.right >= 0 && last + c.right < 0) ||
                    (c.left >= 0 && c.sinks == 0 && c.off - c.left >= Skv);
  if (c.accumulate && none && o_run == nullptr) return CPATTN_OK;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (c.in_f32) return cuda_status(cpattn::launch_window_f32(c, cs));
  if (Skv == 0 && !c.accumulate)
    return cuda_status(cpattn::launch_fill_empty(out, size_t(B) * Sq * H * D * elem_size(out_dtype), lse,
                                                 size_t(B) * H * Sq, cs));
  int* err = cpattn::device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  return cuda_status(cpattn::launch_window_sm100(c, err, cs));
}

int cpattn_window_decode(const void* q, const void* k_cache, const void* v_cache, const int* kv_len,
                         void* out, float* lse, int B, int H, int Hkv, int Sq, int S_max, int D,
                         long long q_stride, long long k_stride, long long v_stride, float scale,
                         int left, int sinks, int in_dtype, int out_dtype, cpattn_stream_t stream) {
  WindowCall c{q, k_cache, v_cache, out, lse, kv_len, nullptr, B, H, Hkv, Sq, S_max, D, q_stride, k_stride,
               v_stride, scale, 0, clamp_extent(left), 0, sinks, true, false, false, false};
  const int st = check(&c, in_dtype, out_dtype);
  if (st != CPATTN_OK) return st;
  if (S_max < 1) return CPATTN_ERR_SHAPE;
  if (sinks > S_max) c.sinks = S_max;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (c.in_f32) return cuda_status(cpattn::launch_window_f32(c, cs));
  if (!tiles_serve(c)) return cuda_status(cpattn::launch_window_decode(c, cs));
  int* err = cpattn::device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  return cuda_status(cpattn::launch_window_sm100(c, err, cs));
}

}  // extern "C"
