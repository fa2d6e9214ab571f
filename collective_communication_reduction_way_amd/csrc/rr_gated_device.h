// rr_gated_device.h -- the activations of the gated projections (gfx950).
#pragma once

#include "rr_device.h"
#include "rr_gated.h"
#include "rr_rows.h"

namespace rr {

// f = act(a) and, where GRAD, df = act'(a).
//   silu: a sig(a), derivative sig (1 + a (1 - sig));
//   gelu: a cdf(a), derivative cdf + a pdf, of the normal distribution.
// 16-bit types: exponentials and reciprocals of the hardware, and for the
// distribution's tail erfc(x) = exp(-x^2) t P(t), t = 1 / (1 + 0.38 x), P fitted to
// erfcx on [0, 10] with a relative error of 1.2e-6, so that small values keep their
// digits and the exponential serves the derivative as well.  float32: the
// library's functions.
template <class E, GatedAct ACT, bool GRAD>
__device__ __forceinline__ float activate(float a, float* df) {
  constexpr bool kFast = sizeof(typename E::S) == 2;
  if constexpr (ACT == GatedAct::kSilu) {
    const float e = 1.f + (kFast ? __expf(-a) : expf(-a));
    const float sig = kFast ? __builtin_amdgcn_rcpf(e) : 1.f / e;
    if constexpr (GRAD) *df = sig * fmaf(a, 1.f - sig, 1.f);
    return a * sig;
  } else {
    constexpr float kRoot = 0.70710678118654752f;  // 1 / sqrt(2)
    const float x = fabsf(a) * kRoot;
    float tail, e = 0.f;  // erfc(|a| / sqrt(2)) / 2
    if constexpr (kFast) {
      const float t = __builtin_amdgcn_rcpf(fmaf(0.38f, x, 1.f));
      e = __expf(-x * x);
      float q = -0.12521542608737946f;
      q = fmaf(q, t, 0.3352506756782532f);
      q = fmaf(q, t, -0.06868264824151993f);
      q = fmaf(q, t, 0.24684418737888336f);
      q = fmaf(q, t, 0.18102401494979858f);
      q = fmaf(q, t, 0.21648254990577698f);
      q = fmaf(q, t, 0.21429559588432312f);
      tail = 0.5f * e * (q * t);
    } else {
      tail = 0.5f * erfcf(x);
      if constexpr (GRAD) e = expf(-0.5f * a * a);
    }
    const float cdf = a < 0.f ? tail : 1.f - tail;
    if constexpr (GRAD) *df = fmaf(a, e * 0.39894228040143268f, cdf);  // 1 / sqrt(2 pi)
    return a * cdf;
  }
}

// The products' gradients in float32: a becomes dA = dh U act'(A), u dU = dh act(A).
// They go to the matrix cores rounded to the storage type, as dh and the weights come: a
// rounding each, of half a step at most.  The results' errors against 64 bits are then those
// of two roundings, 0.0023 in bfloat16 and 0.0003 in float16, where rounding the results alone
// leaves 0.0017 and 0.0002.  To take it back each would have to go as two parts, value and
// remainder, and the gradients' products, three fifths of a long step's time, twice.
template <class E, GatedAct ACT>
__device__ __forceinline__ void gate_grad_one(float dh, float& a, float& u) {
  float df;
  const float f = activate<E, ACT, true>(a, &df);
  a = dh * u * df;
  u = dh * f;
}

// The shard of padded feature f < off[p].
template <class SH>
__device__ __forceinline__ int shard_of(const SH& sh, uint32_t f, int from = 0) {
  int r = from;
  while (f >= sh.off[r + 1]) ++r;  // f < off[p]: ends at the shard that holds f
  return r;
}

// The gate's column of padded feature f in the matrix of both products; up's is
// kFeat further.
__device__ __forceinline__ uint64_t gate_col(uint32_t f) {
  return static_cast<uint64_t>(f / kFeat) * (2 * kFeat) + f % kFeat;
}

// float16 gradients are kept scaled by 2^(15 - e), e the exponent of the row's
// largest finite one (|g| < 2^e), so that a row keeps its digits whatever its
// size and does not leave the type's range; rows without one are not scaled.
__device__ __forceinline__ int row_scale(float row_max) {
  return row_max == 0.f ? 0 : 15 - (ilogbf(row_max) + 1);
}

// N threads, this one `i`, copy row t of x into an aligned one; float16: times
// 2^(e - top + 15), e the exponent of the row's largest gradient (row_scale's) and top
// the largest e + a, |x| < 2^a in a row, so that the rows of grad^T * x have one scale,
// 2^(30 - top), and the largest ends just below 2^15 (token_exponent).
template <class E, uint32_t N>
__device__ __forceinline__ void copy_scaled(const GatedRowsArgs& a, uint64_t t, uint32_t i, int top) {
  using S = typename E::S;
  const S* const x = static_cast<const S*>(a.x) + t * a.dim;
  S* const out = reinterpret_cast<S*>(static_cast<char*>(a.out) + t * a.out_stride);
  float f = 1.f;
  if constexpr (__is_same(E, EF16)) {
    // (a row whose gradients are zeros or infinite ones is as good at any scale)
    const float rm = a.row_max ? a.row_max[t] : 0.f;
    f = rm != 0.f ? row_factor(rm, top) : 1.f;
  }
  for (uint32_t d = i * kEpc<E>; d < a.dim; d += N * kEpc<E>) {
    u32x4 v = load_chunk<E>(x, d, a.dim);
    if constexpr (__is_same(E, EF16)) {
      if (f != 1.f) {
        float w[8];
        widen<E>(v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= f;
        v = narrow<E>(w);
      }
    }
    *reinterpret_cast<u32x4*>(out + d) = v;
  }
}

// dhidden = the splits' sums, rounded once.  A workgroup takes 1024 / G columns of
// row t, four a thread; with G = 4, for many splits, 4 threads share a column's.
// `part`: 1024 floats (G > 1).
template <class E, int G>
__device__ __forceinline__ void join_sums(const GatedJoinArgs& a, uint32_t t, uint32_t by, float* part) {
  using S = typename E::S;
  constexpr uint32_t V = 4, kCols = 256 / G * V;
  const uint32_t c = threadIdx.x % (256 / G), g = threadIdx.x / (256 / G);
  const uint32_t d = by * kCols + c * V;
  float v[V] = {};
  if (d < a.dim) {
    const float* p = a.acc + static_cast<uint64_t>(t) * a.acc_ld + d;
    const uint32_t lo = a.splits * g / G, hi = a.splits * (g + 1) / G;
#pragma unroll 8
    for (uint32_t s = lo; s < hi; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(p + s * a.split_stride);
      v[0] += x.x;
      v[1] += x.y;
      v[2] += x.z;
      v[3] += x.w;
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (uint32_t j = 0; j < V; ++j) part[g * kCols + c * V + j] = v[j];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (uint32_t q = 1; q < G; ++q)
#pragma unroll
      for (uint32_t j = 0; j < V; ++j) v[j] += part[q * kCols + c * V + j];
  }
  float f = 1.f;
  if constexpr (__is_same(E, EF16)) f = ldexpf(1.f, -row_scale(a.row_max[t]));
  S* const out = static_cast<S*>(a.out) + static_cast<uint64_t>(t) * a.dim + d;
#pragma unroll
  for (uint32_t j = 0; j < V; ++j)
    if (d + j < a.dim) store_one<E>(out + j, v[j] * f);
}

}  // namespace rr
