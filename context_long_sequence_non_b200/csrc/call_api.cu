// call_api.cu -- cpattn_call: a call by number with its arguments in 8-byte words (cpattn.h).
#include <cstdint>
#include <cstring>
#include <limits>
#include <tuple>
#include <utility>

#include "cpattn.h"

namespace {

template <class T>
bool read(const unsigned char* word, T** out) {
  uint64_t w;
  std::memcpy(&w, word, 8);
  *out = reinterpret_cast<T*>(static_cast<uintptr_t>(w));
  return true;
}

bool read(const unsigned char* word, long long* out) {
  int64_t w;
  std::memcpy(&w, word, 8);
  *out = w;
  return true;
}

bool read(const unsigned char* word, int* out) {
  long long w;
  read(word, &w);
  *out = static_cast<int>(w);
  return w >= std::numeric_limits<int>::min() && w <= std::numeric_limits<int>::max();
}

bool read(const unsigned char* word, float* out) {
  double w;
  std::memcpy(&w, word, 8);
  *out = static_cast<float>(w);
  return true;
}

template <class... A, size_t... I>
int apply(int (*call)(A...), const unsigned char* words, std::index_sequence<I...>) {
  std::tuple<A...> a;
  if (!(read(words + 8 * I, &std::get<I>(a)) && ...)) return CPATTN_ERR_SHAPE;
  return call(std::get<I>(a)...);
}

template <class... A>
int apply(int (*call)(A...), const unsigned char* words, int n) {
  if (n != int(sizeof...(A))) return CPATTN_ERR_SHAPE;
  return apply(call, words, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" int cpattn_call(int entry, const void* words, int n) {
  if (words == nullptr) return CPATTN_ERR_NULL;
  const unsigned char* w = static_cast<const unsigned char*>(words);
  switch (entry) {
    case CPATTN_CALL_WINDOW_FWD: return apply(cpattn_window_fwd, w, n);
    case CPATTN_CALL_WINDOW_DECODE: return apply(cpattn_window_decode, w, n);
    case CPATTN_CALL_ROPE: return apply(cpattn_rope, w, n);
    case CPATTN_CALL_QK_NORM_ROPE: return apply(cpattn_qk_norm_rope, w, n);
    case CPATTN_CALL_SEQ2HEAD_QKV_NORM_ROPE: return apply(cpattn_seq2head_qkv_norm_rope, w, n);
  }
  return CPATTN_ERR_SHAPE;
}
