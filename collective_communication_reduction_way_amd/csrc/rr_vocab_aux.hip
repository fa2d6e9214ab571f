// rr_vocab_aux.hip -- the vocabulary cross entropy's passes around its matrix
// products: joining the softmax statistics of the vocabulary's tiles, copying
// rows into aligned ones, joining split sums.  All are bound by memory and
// small beside the products.
#include "rr_vocab_device.h"

namespace rr {

namespace {

__device__ __forceinline__ bool counts(const void* targets, int bytes, uint32_t i, uint32_t vocab) {
  const int64_t y = target_at(targets, bytes, i);
  return y >= 0 && y < static_cast<int64_t>(vocab);
}

// lse = log sum exp over the tiles' (maximum, sum) pairs and the loss lse -
// target logit.  P threads share a token, 256 / P tokens a workgroup: 32 where
// there are many tokens (8 tokens' pairs fill a 64-byte segment), 256 where
// there are few (one token's few hundred pairs are read at once: 7.2 -> 3.8 us).
// 8192 tokens and 197 tiles: 8 us.
__device__ __forceinline__ void merge(float& mx, float& sum, float m2, float s2) {
  const float top = fmaxf(mx, m2);
  const float ref = top == -__builtin_inff() ? 0.f : top;
  sum = sum * __expf(mx - ref) + s2 * __expf(m2 - ref);
  mx = top;
}

template <int P>
__global__ __launch_bounds__(256) void k_loss(LossArgs a) {
  constexpr uint32_t T = 256 / P;
  __shared__ float sm[P][T][2];
  const uint32_t ti = threadIdx.x % T, part = threadIdx.x / T;
  const uint32_t t = blockIdx.x * T + ti;
  float mx = -__builtin_inff(), sum = 0.f;
  if (t < a.tokens) {
    const float2* p = reinterpret_cast<const float2*>(a.part) + t;
    uint32_t i = part;
    for (; i + 3 * P < a.tiles; i += 4 * P) {
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = p[static_cast<uint64_t>(i + j * P) * a.tokens];
#pragma unroll
      for (int j = 0; j < 4; ++j) merge(mx, sum, v[j].x, v[j].y);
    }
    for (; i < a.tiles; i += P) {
      const float2 v = p[static_cast<uint64_t>(i) * a.tokens];
      merge(mx, sum, v.x, v.y);
    }
  }
  sm[part][ti][0] = mx;
  sm[part][ti][1] = sum;
  __syncthreads();
  for (uint32_t h = P / 2; h > 0; h >>= 1) {
    if (part < h) {
      merge(mx, sum, sm[part + h][ti][0], sm[part + h][ti][1]);
      sm[part][ti][0] = mx;
      sm[part][ti][1] = sum;
    }
    __syncthreads();
  }
  if (part == 0 && t < a.tokens) {
    const float lse = mx + logf(sum);
    a.lse[t] = lse;
    a.loss[t] = counts(a.targets, a.target_bytes, t, a.vocab) ? lse - a.hit[t] : 0.f;
  }
}

// One workgroup: the largest exponent of the loss gradients that count.
__global__ __launch_bounds__(1024) void k_grad_scale(const float* g, const void* targets, int target_bytes,
                                                     uint32_t tokens, uint32_t vocab, int32_t* scale) {
  __shared__ int sm[16];
  int top = -150;  // below every float32 exponent
  for (uint32_t i = threadIdx.x; i < tokens; i += 1024) {
    const float v = g[i];
    if (v != 0.f && fabsf(v) < __builtin_inff() && counts(targets, target_bytes, i, vocab))
      top = max(top, token_exponent(v));
  }
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) top = max(top, sm[i]);
    *scale = top == -150 ? 0 : top;
  }
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

// A workgroup a row.  Bound by memory: 8192 rows of 4096 bfloat16 values in 23 us
// (5.8 TB/s).
template <class E>
__global__ __launch_bounds__(256) void k_pack_rows(PackRowsArgs a) {
  using S = typename E::S;
  constexpr uint32_t EPC = 16 / sizeof(S);
  const uint32_t t = blockIdx.x;
  uint32_t col = 0;
  if (t < a.tokens && a.targets) {
    col = padded_col(a.sh, target_at(a.targets, a.target_bytes, t));
    if (a.tcol && threadIdx.x == 0) a.tcol[t] = col;
  }
  const bool live = t < a.tokens && col != kMasked;
  float f = 1.f;
  if (a.grad_loss && live) {
    const float g = a.grad_loss[t];
    // a row of g = 0 counts for nothing; one of infinite or NaN g makes the
    // sums that already at scale 1
    f = g == 0.f ? 0.f : fabsf(g) < __builtin_inff() ? ldexpf(1.f, token_exponent(g) - a.scale[0]) : 1.f;
  }
  const S* row = static_cast<const S*>(a.x) + static_cast<uint64_t>(t) * a.dim;
  char* out = static_cast<char*>(a.out) + t * a.out_stride;
  for (uint32_t d = threadIdx.x * EPC; d < a.dim; d += 256 * EPC) {
    __attribute__((aligned(16))) S v[EPC];
    if (live) {
      read_chunk<S>(row, d, a.dim, a.unit, v);
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

template <class S>
__global__ __launch_bounds__(256) void k_pack_weight(PackWeightArgs a) {
  constexpr uint32_t EPC = 16 / sizeof(S);
  const uint32_t c = a.c0 + blockIdx.x;
  const S* row = nullptr;
  for (int r = 0; r < a.sh.p; ++r)
    if (c >= a.sh.off[r] && c - a.sh.off[r] < a.sh.rows[r])
      row = static_cast<const S*>(a.sh.w[r]) + static_cast<uint64_t>(c - a.sh.off[r]) * a.dim;
  char* out = static_cast<char*>(a.out) + blockIdx.x * a.out_stride;
  for (uint32_t d = threadIdx.x * EPC; d < a.dim; d += 256 * EPC) {
    __attribute__((aligned(16))) S v[EPC];
    if (row) {
      read_chunk<S>(row, d, a.dim, a.unit, v);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < EPC; ++j) v[j] = S(0);
    }
    *reinterpret_cast<u32x4*>(out + d * sizeof(S)) = *reinterpret_cast<const u32x4*>(v);
  }
}

// dhidden = the sum of the splits' float32 accumulators, finished and rounded
// once.  A workgroup takes 1024 columns of a row, or 256 where there are many
// splits: then 4 threads share a column's splits, so that a few tokens' few
// columns are not one long chain of loads.
template <class E, int G, int V>
__global__ __launch_bounds__(256) void k_join(JoinArgs a) {
  using S = typename E::S;
  constexpr uint32_t kCols = 256 / G * V;
  __shared__ float part[G][kCols];
  const uint32_t t = blockIdx.x;
  const uint32_t c = threadIdx.x % (256 / G), g = threadIdx.x / (256 / G);
  const uint32_t d = blockIdx.y * kCols + c * V;
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
    for (int j = 0; j < V; ++j) part[g][c * V + j] = v[j];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int q = 1; q < G; ++q)
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += part[q][c * V + j];
  }
  const HiddenRow<E> h(a.sh, a.tcol, a.lo, a.grad_loss, t, a.tokens, a.dim);
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

template <class E>
void run_join(const JoinArgs& a, hipStream_t s) {
  const bool many = a.splits >= 8, vec = a.dim % 4 == 0;
  const uint32_t cols = (many ? 64 : 256) * (vec ? 4 : 1);
  const dim3 g(a.tokens, (a.dim + cols - 1) / cols);
  if (many && vec) hipLaunchKernelGGL((k_join<E, 4, 4>), g, dim3(256), 0, s, a);
  else if (many) hipLaunchKernelGGL((k_join<E, 4, 1>), g, dim3(256), 0, s, a);
  else if (vec) hipLaunchKernelGGL((k_join<E, 1, 4>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_join<E, 1, 1>), g, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_loss(const LossArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  if (a.tokens < 256)
    hipLaunchKernelGGL(k_loss<256>, dim3(a.tokens), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_loss<32>, dim3((a.tokens + 7) / 8), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const float* grad_loss, const void* targets, int target_bytes, uint32_t tokens,
                             uint32_t vocab, int32_t* scale, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_scale, dim3(1), dim3(1024), 0, s, grad_loss, targets, target_bytes, tokens, vocab, scale);
  return hipGetLastError();
}

hipError_t launch_pack_rows(const PackRowsArgs& a, Kind k, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  switch (k) {
    case Kind::kF32: hipLaunchKernelGGL(k_pack_rows<EF32>, dim3(a.rows), dim3(256), 0, s, a); break;
    case Kind::kBF16: hipLaunchKernelGGL(k_pack_rows<EBF16>, dim3(a.rows), dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL(k_pack_rows<EF16>, dim3(a.rows), dim3(256), 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_pack_weight(const PackWeightArgs& a, Kind k, hipStream_t s) {
  const dim3 g(a.c1 - a.c0);
  if (k == Kind::kF32)
    hipLaunchKernelGGL(k_pack_weight<uint32_t>, g, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_pack_weight<uint16_t>, g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_join(const JoinArgs& a, Kind k, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  switch (k) {
    case Kind::kF32: run_join<EF32>(a, s); break;
    case Kind::kBF16: run_join<EBF16>(a, s); break;
    default: run_join<EF16>(a, s); break;
  }
  return hipGetLastError();
}

#define RR_DISPATCH(CALL)                 \
  switch (k) {                            \
    case Kind::kF32: return CALL(f32);    \
    case Kind::kBF16: return CALL(bf16);  \
    default: return CALL(f16);            \
  }

hipError_t launch_logits(const LogitArgs& a, Kind k, VocabTile t, bool grad, hipStream_t s) {
#define RR_CALL(NAME) launch_logits_##NAME(a, t, grad, s)
  RR_DISPATCH(RR_CALL)
#undef RR_CALL
}
hipError_t launch_hidden_grad(const HiddenGradArgs& a, Kind k, VocabTile t, hipStream_t s) {
#define RR_CALL(NAME) launch_hidden_grad_##NAME(a, t, s)
  RR_DISPATCH(RR_CALL)
#undef RR_CALL
}
hipError_t launch_weight_grad(const WeightGradArgs& a, Kind k, VocabTile t, hipStream_t s) {
#define RR_CALL(NAME) launch_weight_grad_##NAME(a, t, s)
  RR_DISPATCH(RR_CALL)
#undef RR_CALL
}

}  // namespace rr
