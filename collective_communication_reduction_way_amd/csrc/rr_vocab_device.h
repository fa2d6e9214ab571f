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

}  // namespace rr
