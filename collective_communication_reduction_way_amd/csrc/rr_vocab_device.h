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
// about 2^-29 stay normal numbers.  The hidden rows of dweights then have to be
// scaled by 2^e and a factor that all tokens share: 2^(e - m + 15), where m is the
// largest e + a of the tokens that count and |h| < 2^a in a token's row, so that
// the largest row ends just below 2^15.  What lies below 2^-14 after that, less
// than 2^-29 of the largest |g| |h|, is rounded to a multiple of 2^-24: off by at most
// 2^-38 of that largest product, far below the float32 sum of a row that it is
// part of.  (Scaled by 2^(e - e_max) alone, values of 0.02 lost 11 % at a g of 2^-16
// of the largest.)
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

__device__ __forceinline__ bool counts(const void* targets, int bytes, uint32_t i, uint32_t vocab) {
  const int64_t y = target_at(targets, bytes, i);
  return y >= 0 && y < static_cast<int64_t>(vocab);
}

// m of the tokens' e + a (k_row_exponent), by a workgroup of N threads; 0 where
// none counts.  sm: N / 64 words.
constexpr int kNoExponent = -1000;  // below every e + a
template <int N>
__device__ __forceinline__ int top_exponent(const int32_t* row_exp, uint32_t tokens, int* sm) {
  int top = kNoExponent;
  for (uint32_t i = threadIdx.x; i < tokens; i += N) top = max(top, row_exp[i]);
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = top;
  __syncthreads();
  for (int i = 0; i < N / 64; ++i) top = max(top, sm[i]);
  return top == kNoExponent ? 0 : top;
}

// The factor of a hidden row in float16's dweights.  A row of g = 0 counts for
// nothing; one of infinite or NaN g makes the sums that already at scale 1; one
// without a finite value other than 0 is not in `top`, and its factor stays finite.
__device__ __forceinline__ float row_factor(float g, int top) {
  return g == 0.f ? 0.f : fabsf(g) < __builtin_inff() ? ldexpf(1.f, min(token_exponent(g) - top + 15, 100)) : 1.f;
}

// 16 bytes of a row from element d on, zeros from `dim` on; in loads of `unit`
// bytes where the row goes on that far.
template <class S>
__device__ __forceinline__ void read_chunk(const S* row, uint32_t d, uint32_t dim, uint32_t unit, S* out) {
  constexpr uint32_t EPC = 16 / sizeof(S);
  const bool whole = d + EPC <= dim;
  if (whole && unit == 16) {
    *reinterpret_cast<u32x4*>(out) = *reinterpret_cast<const u32x4*>(row + d);
  } else if (whole && unit == 8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) reinterpret_cast<uint2*>(out)[j] = reinterpret_cast<const uint2*>(row + d)[j];
  } else if (whole && unit == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(out)[j] = reinterpret_cast<const uint32_t*>(row + d)[j];
  } else {
#pragma unroll
    for (uint32_t j = 0; j < EPC; ++j) out[j] = d + j < dim ? row[d + j] : S(0);
  }
}

// N threads, this one `i`, copy a row of dim elements, times f in float16, to
// 16-byte chunks; zeros if it is not live.
template <class E, uint32_t N>
__device__ __forceinline__ void copy_row(const typename E::S* row, char* out, uint32_t dim, uint32_t unit, uint32_t i,
                                         bool live, float f) {
  using S = typename E::S;
  constexpr uint32_t EPC = 16 / sizeof(S);
  for (uint32_t d = i * EPC; d < dim; d += N * EPC) {
    __attribute__((aligned(16))) S v[EPC];
    if (live) {
      read_chunk<S>(row, d, dim, unit, v);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < EPC; ++j) v[j] = S(0);
    }
    if constexpr (__is_same(E, EF16)) {
      if (f != 1.f) {
#pragma unroll
        for (uint32_t j = 0; j < EPC; ++j) v[j] = static_cast<S>(f32_to_f16_bits(f16_bits_to_f32(v[j]) * f));
      }
    }
    *reinterpret_cast<u32x4*>(out + d * sizeof(S)) = *reinterpret_cast<const u32x4*>(v);
  }
}

// dhidden = the sum of the splits' float32 accumulators, finished and rounded
// once.  A workgroup takes 1024 columns of a row, or 256 where there are many
// splits: then 4 threads share a column's splits, so that a few tokens' few
// columns are not one long chain of loads.  `part`: 256 V floats (G > 1).
template <class E, int G, int V>
__device__ __forceinline__ void join_block(const VocabShards& sh, const JoinPart& a, uint32_t t, uint32_t by,
                                           float* part) {
  using S = typename E::S;
  constexpr uint32_t kCols = 256 / G * V;
  const uint32_t c = threadIdx.x % (256 / G), g = threadIdx.x / (256 / G);
  const uint32_t d = by * kCols + c * V;
  const uint64_t at = static_cast<uint64_t>(t) * a.dim + d;
  float v[V] = {};
  if (d < a.dim) {
    const float* p = a.acc + at;
    const uint32_t lo = a.splits * g / G, hi = a.splits * (g + 1) / G;
#pragma unroll 8
    for (uint32_t s = lo; s < hi; ++s) {
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + s * a.split_stride);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      } else {
        v[0] += p[s * a.split_stride];
      }
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) part[g * kCols + c * V + j] = v[j];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int q = 1; q < G; ++q)
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += part[q * kCols + c * V + j];
  }
  const HiddenRow<E> h(sh, a.tcol, a.lo, a.grad_loss, t, a.tokens, a.dim);
  S* out = static_cast<S*>(a.out) + at;
  if constexpr (V == 4 && sizeof(S) == 2) {
    if (a.vec) {
      if (d >= a.dim) return;
      h.finish4(v, d, a.dim);
      uint2 w = make_uint2(0, 0);
      if (h.live) {
        if constexpr (__is_same(E, EBF16))
          w = make_uint2(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]));
        else
          w = make_uint2(f32x2_to_f16x2_bits(v[0], v[1]), f32x2_to_f16x2_bits(v[2], v[3]));
      }
      *reinterpret_cast<uint2*>(out) = w;
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (d + j >= a.dim) break;
    float w = 0.f;
    if constexpr (sizeof(S) == 2) w = h.live ? load_one<E>(h.w + d + j) : 0.f;
    store_one<E>(out + j, h.live ? h.finish(v[j], w) : 0.f);
  }
}

}  // namespace rr
