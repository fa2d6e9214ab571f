// rr_vocab_device.h -- device helpers shared by the vocabulary cross entropy's
// kernels.
#pragma once

#include "rr_device.h"
#include "rr_vocab.h"

namespace rr {

__device__ __forceinline__ int64_t target_at(const void* t, int bytes, uint32_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(t)[i] : static_cast<const int32_t*>(t)[i];
}

// The padded column of vocabulary row y, or kMasked for a masked token (y
// outside the vocabulary).
__device__ __forceinline__ uint32_t padded_col(const VocabShards& sh, int64_t y) {
  if (y < 0 || y >= static_cast<int64_t>(sh.vocab)) return kMasked;
  const uint32_t v = static_cast<uint32_t>(y);
  uint32_t c = 0;
  for (int r = 0; r < sh.p; ++r)
    if (v >= sh.first[r] && v - sh.first[r] < sh.rows[r]) c = sh.off[r] + (v - sh.first[r]);
  return c;
}

// float16 scaling by powers of two.  The gradient of a token's logits is kept
// as (p - onehot) * g * 2^(15 - e), e the exponent with |g| < 2^e, so that a row
// keeps its precision whatever the size of its g and probabilities down to
// about 2^-29 stay normal numbers; the hidden rows of dweights are scaled by
// 2^(e - e_max).  Neither scaling rounds (the hidden rows only where they
// become subnormal: tokens that count 2^-10 of the largest or less).
__device__ __forceinline__ int token_exponent(float g) {
  if (!(fabsf(g) < __builtin_inff()) || g == 0.f) return 0;  // inf, NaN and 0 scale to themselves
  return ilogbf(g) + 1;
}

// What a row of dhidden gets besides its product: the rounding remainder of
// the target's entry times the target's weights (16-bit types), and the row's
// scale (float16).  A masked token's row is zero whatever the weights hold.
template <class E>
struct HiddenRow {
  using S = typename E::S;
  const S* w = nullptr;  // the target's weights
  float lo = 0.f, f = 1.f;
  bool live = false;

  __device__ __forceinline__ HiddenRow(const VocabShards& sh, const uint32_t* tcol, const float* lo_, const float* g,
                                       uint32_t t, uint32_t tokens, uint32_t dim) {
    const uint32_t col = t < tokens ? tcol[t] : kMasked;
    live = col != kMasked;
    if (!live) return;
    if constexpr (__is_same(E, EF16)) f = ldexpf(1.f, token_exponent(g[t]) - 15);
    if constexpr (sizeof(S) == 2) {
      lo = lo_[t];
      for (int r = 0; r < sh.p; ++r)
        if (col >= sh.off[r] && col - sh.off[r] < sh.rows[r])
          w = static_cast<const S*>(sh.w[r]) + static_cast<uint64_t>(col - sh.off[r]) * dim;
    }
  }
  __device__ __forceinline__ float finish(float v, float weight) const {
    if constexpr (sizeof(S) == 2) v = fmaf(lo, weight, v);
    if constexpr (__is_same(E, EF16)) v *= f;
    return v;
  }
  // Elements d .. d+3 of a row whose weights are 8-byte aligned (16-bit types).
  __device__ __forceinline__ void finish4(float* v, uint32_t d, uint32_t dim) const {
    if (!live || d >= dim) return;
    const uint2 x = *reinterpret_cast<const uint2*>(w + d);
    v[0] = finish(v[0], half_to_f32<E>(x.x & 0xFFFFu));
    v[1] = finish(v[1], half_to_f32<E>(x.x >> 16));
    v[2] = finish(v[2], half_to_f32<E>(x.y & 0xFFFFu));
    v[3] = finish(v[3], half_to_f32<E>(x.y >> 16));
  }
};

}  // namespace rr
