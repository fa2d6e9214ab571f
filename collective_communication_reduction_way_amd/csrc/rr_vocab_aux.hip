// rr_vocab_aux.hip -- the vocabulary cross entropy's passes around its matrix
// products: joining the softmax statistics of the vocabulary's tiles, copying
// rows into aligned ones, joining split sums.  All are bound by memory and
// small beside the products.
#include "rr_vocab_device.h"

namespace rr {

namespace {

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

// A workgroup a row: the exponents of its loss gradient and of its largest
// finite hidden value, as integers.  One read of the hidden states (96 x 768: 3 us
// of a step of 119).
__global__ __launch_bounds__(256) void k_row_exponent(RowExponentArgs a) {
  constexpr uint32_t EPC = 8;
  __shared__ uint32_t sm[4];
  const uint32_t t = blockIdx.x;
  const float g = a.grad_loss[t];
  int e = kNoExponent;
  if (g != 0.f && fabsf(g) < __builtin_inff() && counts(a.targets, a.target_bytes, t, a.vocab)) {
    const uint16_t* row = static_cast<const uint16_t*>(a.x) + static_cast<uint64_t>(t) * a.dim;
    uint32_t top = 0;
    for (uint32_t d = threadIdx.x * EPC; d < a.dim; d += 256 * EPC) {
      __attribute__((aligned(16))) uint16_t v[EPC];
      read_chunk<uint16_t>(row, d, a.dim, a.unit, v);
#pragma unroll
      for (uint32_t j = 0; j < EPC; ++j) {
        const uint32_t b = v[j] & 0x7FFFu;
        top = max(top, b < 0x7C00u ? b : 0u);
      }
    }
    for (int o = 32; o > 0; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, sm[i]);
    if (top) e = token_exponent(g) + ilogbf(f16_bits_to_f32(top)) + 1;
  }
  if (threadIdx.x == 0) a.out[t] = e;
}

// One workgroup: the largest of the rows' exponents.
__global__ __launch_bounds__(1024) void k_grad_scale(const int32_t* row_exp, uint32_t tokens, int32_t* scale) {
  __shared__ int sm[16];
  const int top = top_exponent<1024>(row_exp, tokens, sm);
  if (threadIdx.x == 0) *scale = top;
}

// A workgroup a row.  Bound by memory: 8192 rows of 4096 bfloat16 values in 23 us
// (5.8 TB/s).
template <class E>
__global__ __launch_bounds__(256) void k_pack_rows(PackRowsArgs a) {
  using S = typename E::S;
  const uint32_t t = blockIdx.x;
  uint32_t col = 0;
  if (t < a.tokens && a.targets) {
    col = padded_col(a.sh, target_at(a.targets, a.target_bytes, t));
    if (a.tcol && threadIdx.x == 0) a.tcol[t] = col;
  }
  const bool live = t < a.tokens && col != kMasked;
  const float f = a.grad_loss && live ? row_factor(a.grad_loss[t], a.scale[0]) : 1.f;
  copy_row<E, 256>(static_cast<const S*>(a.x) + static_cast<uint64_t>(t) * a.dim,
                   static_cast<char*>(a.out) + t * a.out_stride, a.dim, a.unit, threadIdx.x, live, f);
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

template <class E, int G, int V>
__global__ __launch_bounds__(256) void k_join(JoinArgs a) {
  __shared__ float part[G > 1 ? 256 * V : 1];
  join_block<E, G, V>(a.sh, a, blockIdx.x, blockIdx.y, part);
}

template <class E>
void run_join(const JoinArgs& a, hipStream_t s) {
  const bool many = a.splits >= kJoinMany, vec = a.dim % 4 == 0;
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

hipError_t launch_row_exponent(const RowExponentArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  hipLaunchKernelGGL(k_row_exponent, dim3(a.tokens), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const int32_t* row_exp, uint32_t tokens, int32_t* scale, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_scale, dim3(1), dim3(1024), 0, s, row_exp, tokens, scale);
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
