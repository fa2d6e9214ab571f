// rr_norm.hip -- layer norm and root-mean-square norm over the ranks' rows, and
// their gradients (gfx950).
//
//   y = xh w + b,  xh = (x - m) s,  s = 1 / sqrt(v + eps);  m and v a row's mean
//   and variance, or 0 and its mean square;
//   dx = s (g - mean(g) - xh mean(g xh)) + residual,  g = dy w (the root-mean-
//   square norm has no mean(g));  dw = sum dy xh,  db = sum dy over all rows.
//
// A row is read once: W wavefronts hold it in registers, K chunks of 16 bytes a
// lane, in the storage type.  The mean's rounding is taken off again in a second
// look at the registers, where the variance is summed about the mean: no
// difference of large sums is formed.  Both directions are bound by memory.
#include "rr_device.h"
#include "rr_norm.h"
#include "rr_rows.h"

namespace rr {

namespace {

// The sum over a wavefront, in every lane.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);   // lane xor 1
  v += dpp<0x4E>(v);   // lane xor 2
  v += dpp<0x141>(v);  // the other four of eight
  v += dpp<0x140>(v);  // the other eight of sixteen
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sums of N <= 2 values over the W wavefronts that share a row; sm: 4 W floats of the row,
// used in turn so that one barrier a sum is enough.
template <int W, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sm, uint32_t& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    float* const q = sm + (turn & 1) * 2 * W;
    ++turn;
    const int wave = (threadIdx.x >> 6) % W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i * W + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += q[i * W + w];
      v[i] = t;
    }
  }
}

// A row goes to W wavefronts, K chunks a lane, by its 16-byte chunks.  Few chunks a
// lane keep many rows in flight and few registers in use: rows of 4096 bfloat16
// values, 8 x 2048 of them, forward with one wavefront a row and 8 chunks a lane
// 82 us, with four and 2 chunks 45 (5.9 TB/s; a copy of this library 6.4);
// gradient with residuals 122 and, with eight and one chunk, 87 us (6.2 TB/s; without
// residuals 70); 16384 rows of 1024, with one wavefront and 2 chunks 31 us, with two and one
// chunk 28.
struct Shape {
  int w, k;
};
constexpr int kGradWaves = 8;  // of a workgroup of the gradient: 8 / W rows at once
constexpr int forward_rows(int W) { return W == 1 ? 4 : 1; }

// Nontemporal stores: what is written is not read here again (rows of 768, 8192 of
// them: 7.6 -> 6.4 us); nontemporal loads gain in the gradient only (W = 8, with
// residuals: 95 -> 89 us), where three streams are read.
//
// A row's last chunk.  No load is conditional: what a branch may skip the compiler has
// to wait for at once.  A lane whose chunk does not lie in the row whole reads the row's
// last 16 bytes, and what it reads twice is shifted out where the chunk is used (gradient
// with residuals, matrices of the size of 15000 x 4096, TB/s, with branches / so: 3000 bfloat16
// values 2.9 / 4.0, 4095 1.9 / 3.7, 4438 1.4 / 3.3, 1023 float32 ones 3.6 / 5.0).  Rows of less
// than 16 bytes are read by elements, and the gradient's 8 chunks a lane, which have no registers
// to spare, with branches (BRANCH).
template <class E, bool BRANCH>
__device__ __forceinline__ uint32_t chunk_at(uint32_t e, uint32_t dim) {  // bytes into the row, or the element (BRANCH)
  if constexpr (BRANCH) return e;
  const uint32_t last = dim - kEpc<E>;
  return (e < last ? e : last) * static_cast<uint32_t>(sizeof(typename E::S));
}
template <class E, bool BRANCH, bool STREAM>
__device__ __forceinline__ u32x4 fetch_chunk(const typename E::S* row, uint32_t at, uint32_t dim) {
  if constexpr (BRANCH) {
    if (STREAM && at + kEpc<E> <= dim) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + at));
    return load_chunk<E>(row, at, dim);
  }
  const u32x4_any* const p = reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(row) + at);
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}
// The chunk at element e of what fetch_chunk read for it, zeros from dim on; `end`: past the
// wavefronts' last element of this chunk.
template <class E, bool BRANCH>
__device__ __forceinline__ void settle(u32x4& r, uint32_t e, uint32_t end, uint32_t dim) {
  if (BRANCH || end <= dim) return;
  constexpr uint32_t V = kEpc<E>;
  const uint32_t over = e + V > dim ? (e + V - dim < V ? e + V - dim : V) : 0;  // elements
  if constexpr (V == 8) {
    if (dim % 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = r[i] >> 16 | (i < 3 ? r[i + 1] << 16 : 0u);
        r[i] = over & 1 ? w : r[i];
      }
    }
  }
  const uint32_t words = V == 8 ? over / 2 : over;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = words & 1 ? (i < 3 ? r[i + 1] : 0u) : r[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = words & 2 ? (i < 2 ? r[i + 2] : 0u) : r[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = words & 4 ? 0u : r[i];
}
template <class E>
__device__ __forceinline__ void put_chunk(typename E::S* row, uint32_t e, uint32_t dim, u32x4 v) {
  if (e + kEpc<E> <= dim)
    __builtin_nontemporal_store(static_cast<u32x4_any>(v), reinterpret_cast<u32x4_any*>(row + e));
  else
    store_chunk<E>(row, e, dim, v);
}

template <class E, int W, int K, bool BRANCH>
__global__ __launch_bounds__(64 * W * forward_rows(W)) void k_norm(NormArgs a) {
  using S = typename E::S;
  constexpr int V = kEpc<E>;
  constexpr uint32_t kStep = 64u * W * V;
  __shared__ float sm[4 * W];
  uint32_t turn = 0;
  const uint32_t lane = threadIdx.x % (64 * W);
  const uint32_t e0 = lane * V;
  uint32_t off[K];
#pragma unroll
  for (int k = 0; k < K; ++k) off[k] = chunk_at<E, BRANCH>(e0 + k * kStep, a.dim);
  const float inv = 1.f / static_cast<float>(a.dim);
  const uint32_t cut = a.dim % V ? a.dim : ~0u;  // chunks that lie in part in the row
  // (wavefronts past the row's end load nothing: where a row has one turn that is worth the
  // branch, 7492 rows of 8200 bfloat16 values 113 -> 102 us)
  const auto get = [&](const S* row, int k) __attribute__((always_inline)) {
    u32x4 r = {0, 0, 0, 0};
    if (e0 + k * kStep < a.dim) r = fetch_chunk<E, BRANCH, false>(row, off[k], a.dim);
    return r;
  };
  for (uint32_t i = blockIdx.x * forward_rows(W) + __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * W)); i < a.total;
       i += gridDim.x * forward_rows(W)) {
    const uint32_t r = i / a.rows;
    const uint64_t at = static_cast<uint64_t>(i - r * a.rows) * a.dim;
    const S* const x = static_cast<const S*>(a.in[r]) + at;
    u32x4 raw[K], wr[K], br[K];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k] = get(x, k);
    if (a.weight) {
#pragma unroll
      for (int k = 0; k < K; ++k) wr[k] = get(static_cast<const S*>(a.weight), k);
    }
    if (a.bias) {
#pragma unroll
      for (int k = 0; k < K; ++k) br[k] = get(static_cast<const S*>(a.bias), k);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) settle<E, BRANCH>(raw[k], e0 + k * kStep, (k + 1) * kStep, cut);
    float m = 0.f;
    if (a.center) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[V];
        widen<E>(raw[k], v);
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] += v[j];
      }
      row_sum<W>(s, sm, turn);
      m = s[0] * inv;
    }
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V];
      widen<E>(raw[k], v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] -= m;
      if ((k + 1) * kStep > a.dim) {  // what lies past the row's end is no value of it
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = e0 + k * kStep + j < a.dim ? v[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        q[0] += v[j];
        q[1] = fmaf(v[j], v[j], q[1]);
      }
    }
    q[1] *= a.fit;
    row_sum<W>(q, sm, turn);
    q[1] *= inv * a.back;
    const float c = a.center ? q[0] * inv : 0.f;
    const float var = a.center ? fmaxf(fmaf(-c, c, q[1]), 0.f) : q[1];
    const float rstd = 1.f / sqrtf(var + a.eps);
    S* const y = static_cast<S*>(a.out[r]) + at;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V], w[V], b[V];
      widen<E>(raw[k], v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = (v[j] - m - c) * rstd;
      if (a.weight) {
        settle<E, BRANCH>(wr[k], e0 + k * kStep, (k + 1) * kStep, cut);
        widen<E>(wr[k], w);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= w[j];
      }
      if (a.bias) {
        settle<E, BRANCH>(br[k], e0 + k * kStep, (k + 1) * kStep, cut);
        widen<E>(br[k], b);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += b[j];
      }
      put_chunk<E>(y, e0 + k * kStep, a.dim, narrow<E>(v));
    }
    if (lane == 0) {
      if (a.mean) a.mean[i] = m + c;
      if (a.rstd) a.rstd[i] = rstd;
    }
  }
}

// The gradient.  A workgroup walks its rows with the sums of dy xh and dy of its
// columns in registers, the next row's loads in flight while one is worked on;
// at the end the rows that went side by side are added in LDS, and one line of
// sums a workgroup leaves for k_norm_join.
template <class E, int W, int K, bool BRANCH>
__global__ __launch_bounds__(64 * kGradWaves) void k_norm_grad(NormGradArgs a) {
  using S = typename E::S;
  constexpr int V = kEpc<E>, G = kGradWaves / W;
  constexpr uint32_t kStep = 64u * W * V;
  constexpr bool kAhead = K <= 4;  // (8 chunks of three streams twice would not fit the registers)
  __shared__ __attribute__((aligned(16))) float sm[G > 1 ? G * kStep : 1];
  __shared__ float sr[G][4 * W];
  uint32_t turn = 0;
  const uint32_t lane = threadIdx.x % (64 * W);
  const uint32_t group = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * W));
  const uint32_t e0 = lane * V;
  uint32_t off[K];
#pragma unroll
  for (int k = 0; k < K; ++k) off[k] = chunk_at<E, BRANCH>(e0 + k * kStep, a.dim);
  const float inv = 1.f / static_cast<float>(a.dim);
  u32x4 wr[K];
  if (a.weight) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      wr[k] = fetch_chunk<E, BRANCH, false>(static_cast<const S*>(a.weight), off[k], a.dim);
      settle<E, BRANCH>(wr[k], e0 + k * kStep, (k + 1) * kStep, a.dim);
    }
  } else {
    float one[V];
#pragma unroll
    for (int j = 0; j < V; ++j) one[j] = 1.f;
#pragma unroll
    for (int k = 0; k < K; ++k) wr[k] = narrow<E>(one);
  }
  float dw[K][V] = {}, db[K][V] = {};
  u32x4 xn[K], gn[K], zn[K];
  float mn = 0.f, sn = 0.f;
  const auto fetch = [&](uint32_t i) __attribute__((always_inline)) {
    if constexpr (kAhead) {
      if (i >= a.total) return;
    } else {
      i = i < a.total ? i : a.total - 1;  // past the end: the last row, unused
    }
    const uint32_t r = i / a.rows;
    const uint64_t at = static_cast<uint64_t>(i - r * a.rows) * a.dim;
    if (a.center) mn = a.mean[i];
    sn = a.rstd[i];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xn[k] = fetch_chunk<E, BRANCH, true>(static_cast<const S*>(a.x[r]) + at, off[k], a.dim);
      gn[k] = fetch_chunk<E, BRANCH, true>(static_cast<const S*>(a.dy[r]) + at, off[k], a.dim);
    }
    if (a.has_res) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        zn[k] = fetch_chunk<E, BRANCH, true>(static_cast<const S*>(a.res[r]) + at, off[k], a.dim);
    }
  };
  const uint32_t step = gridDim.x * G;
  if constexpr (kAhead) fetch(blockIdx.x * G + group);
  for (uint32_t i0 = blockIdx.x * G; i0 < a.total; i0 += step) {  // the same number of turns for every group
    const uint32_t i = i0 + group;
    const bool live = i < a.total;
    if constexpr (!kAhead) fetch(i);
    u32x4 xr[K], gr[K], zr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xr[k] = xn[k];
      gr[k] = gn[k];
      zr[k] = zn[k];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      settle<E, BRANCH>(xr[k], e0 + k * kStep, (k + 1) * kStep, a.dim);
      settle<E, BRANCH>(gr[k], e0 + k * kStep, (k + 1) * kStep, a.dim);
    }
    const float m = mn, rstd = sn;
    // (in place: a row that is written belongs to this group, the next one's is another)
    if constexpr (kAhead) fetch(i + step);
    float s[2] = {0.f, 0.f};
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[V], g[V], w[V];
        widen<E>(xr[k], v);
        widen<E>(gr[k], g);  // zeros past the row's end
        widen<E>(wr[k], w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (v[j] - m) * rstd;
          dw[k][j] = fmaf(g[j], xh, dw[k][j]);
          db[k][j] += g[j];
          const float gw = g[j] * w[j];
          s[0] += gw;
          s[1] = fmaf(gw, xh, s[1]);
        }
      }
    }
    if (!a.has_dx) continue;
    row_sum<W>(s, sr[group], turn);
    if (!live) continue;
    const float s0 = a.center ? s[0] * inv : 0.f, s1 = s[1] * inv;
    const uint32_t r = i / a.rows;
    S* const dx = static_cast<S*>(a.dx[r]) + static_cast<uint64_t>(i - r * a.rows) * a.dim;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V], g[V], w[V];
      widen<E>(xr[k], v);
      widen<E>(gr[k], g);
      widen<E>(wr[k], w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (v[j] - m) * rstd;
        v[j] = (fmaf(g[j], w[j], -s0) - xh * s1) * rstd;
      }
      if (a.has_res) {
        float z[V];
        settle<E, BRANCH>(zr[k], e0 + k * kStep, (k + 1) * kStep, a.dim);
        widen<E>(zr[k], z);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += z[j];
      }
      put_chunk<E>(dx, e0 + k * kStep, a.dim, narrow<E>(v));
    }
  }
  if (!a.part) return;
  const uint32_t ld = (a.dim + 3) / 4 * 4;
  float* const part = a.part + static_cast<uint64_t>(blockIdx.x) * norm_line(a.dim);
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float* const to = G > 1 ? sm + group * kStep + e0 : part + side * ld + k * kStep + e0;
      if constexpr (G > 1) __syncthreads();
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float* const v = (side ? db[k] : dw[k]) + j;
        if (G > 1 || k * kStep + e0 + j < ld) *reinterpret_cast<float4*>(to + j) = make_float4(v[0], v[1], v[2], v[3]);
      }
      if constexpr (G > 1) {
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < kStep && k * kStep + c < ld; c += 64 * kGradWaves) {
          float t = sm[c];
#pragma unroll
          for (int g = 1; g < G; ++g) t += sm[g * kStep + c];
          part[side * ld + k * kStep + c] = t;
        }
      }
    }
}

// dweight and dbias: 16 columns a workgroup, 64 threads share four columns' parts, so
// that 512 parts are one round of loads (512 parts of 4096 columns, both sums: 5 us).
template <class E>
__global__ __launch_bounds__(256) void k_norm_join(NormJoinArgs a) {
  using S = typename E::S;
  constexpr uint32_t C = 4, G = 64;  // groups of 4 columns, threads that share one
  __shared__ float4 sm[G][C];
  const uint32_t ld = (a.dim + 3) / 4 * 4;
  const uint32_t c = threadIdx.x % C, g = threadIdx.x / C;
  const uint32_t e = (blockIdx.x * C + c) * 4;
  const uint32_t which = a.dweight ? blockIdx.y : 1;  // 0: dweight, 1: dbias
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (e < ld) {
    const float* p = a.part + which * ld + e;
#pragma unroll 8
    for (uint32_t i = g; i < a.parts; i += G) {
      const float4 v = *reinterpret_cast<const float4*>(p + static_cast<uint64_t>(i) * norm_line(a.dim));
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
  }
  sm[g][c] = t;
  __syncthreads();
  // 16 columns of 64 sums each: 16 threads a column
  const uint32_t col = threadIdx.x / 16, part = threadIdx.x % 16;
  const float* q = reinterpret_cast<const float*>(sm) + col;
  float sum = 0.f;
#pragma unroll
  for (uint32_t i = 0; i < G / 16; ++i) sum += q[(i * 16 + part) * 16];
  sum += dpp<0xB1>(sum);
  sum += dpp<0x4E>(sum);
  sum += dpp<0x141>(sum);
  sum += dpp<0x140>(sum);
  const uint32_t d = blockIdx.x * 16 + col;
  if (part == 0 && d < a.dim) store_one<E>(static_cast<S*>(which ? a.dbias : a.dweight) + d, sum);
}

uint32_t chunks_of(uint32_t dim, Kind k) { return k == Kind::kF32 ? (dim + 3) / 4 : (dim + 7) / 8; }

Shape forward_shape(uint32_t dim, Kind k) {
  const uint32_t c = chunks_of(dim, k);
  return c <= 64 ? Shape{1, 1} : c <= 128 ? Shape{1, 2} : c <= 256 ? Shape{4, 1} : c <= 512 ? Shape{4, 2}
       : c <= 1024 ? Shape{8, 2} : c <= 2048 ? Shape{8, 4} : Shape{8, 8};
}

Shape grad_shape(uint32_t dim, Kind k) {
  const uint32_t c = chunks_of(dim, k);
  return c <= 64 ? Shape{1, 1} : c <= 128 ? Shape{2, 1} : c <= 256 ? Shape{4, 1} : c <= 512 ? Shape{8, 1}
       : c <= 1024 ? Shape{8, 2} : c <= 2048 ? Shape{8, 4} : Shape{8, 8};
}

constexpr uint32_t kNormGrid = 1u << 20;  // workgroups of the forward pass at most
// Of the gradient, two a compute unit where their lines of sums are little beside the
// rows (a tenth; both go with the row's length, so that the rows decide), else one, and
// rows evenly over them.  Without residuals, with the join, 512 / 256 workgroups, us: bfloat16,
// 16384 rows of 4096 79 / 83 (1024: 87), 4096 rows 33 / 32, 2048 rows 26 / 23, 300 rows 15 with 256 and 12
// with 150; 2000 rows of 2048 16.2 / 13.8; 4096 rows of 1024 12.7 / 11.4; 8192 rows of 768
// 17.3 / 20.0; 999 float32 rows of 1023 11.8 / 10.3, 4096 of 768 15.0 / 16.0.
constexpr uint32_t kNormGradGrid = 512;
constexpr uint32_t kManyRowBytes = 12288;  // a column's

template <class E>
hipError_t run_norm(const NormArgs& a, Shape sh, hipStream_t s) {
  const uint32_t per = forward_rows(sh.w), need = (a.total + per - 1) / per;
  const dim3 g(need < kNormGrid ? need : kNormGrid);
  if (a.dim < kEpc<E>) {
    hipLaunchKernelGGL((k_norm<E, 1, 1, true>), g, dim3(64 * forward_rows(1)), 0, s, a);
    return hipGetLastError();
  }
#define RR_NORM(W, K)                                                                         \
  if (sh.w == W && sh.k == K) {                                                               \
    hipLaunchKernelGGL((k_norm<E, W, K, false>), g, dim3(64 * W * forward_rows(W)), 0, s, a); \
    return hipGetLastError();                                                                 \
  }
  RR_NORM(1, 1)
  RR_NORM(1, 2)
  RR_NORM(4, 1)
  RR_NORM(4, 2)
  RR_NORM(8, 2)
  RR_NORM(8, 4)
  if constexpr (sizeof(typename E::S) == 4) {
    RR_NORM(8, 8)
  }
#undef RR_NORM
  return hipErrorInvalidValue;
}

template <class E>
hipError_t run_norm_grad(const NormGradArgs& a, Shape sh, uint32_t grid, hipStream_t s) {
  if (a.dim < kEpc<E>) {
    hipLaunchKernelGGL((k_norm_grad<E, 1, 1, true>), dim3(grid), dim3(64 * kGradWaves), 0, s, a);
    return hipGetLastError();
  }
#define RR_NORM(W, K)                                                                              \
  if (sh.w == W && sh.k == K) {                                                                    \
    hipLaunchKernelGGL((k_norm_grad<E, W, K, (K > 4)>), dim3(grid), dim3(64 * kGradWaves), 0, s, a); \
    return hipGetLastError();                                                                      \
  }
  RR_NORM(1, 1)
  RR_NORM(2, 1)
  RR_NORM(4, 1)
  RR_NORM(8, 1)
  RR_NORM(8, 2)
  RR_NORM(8, 4)
  if constexpr (sizeof(typename E::S) == 4) {
    RR_NORM(8, 8)
  }
#undef RR_NORM
  return hipErrorInvalidValue;
}

}  // namespace

uint32_t norm_grad_grid(uint32_t total, uint32_t dim, Kind k) {
  const uint32_t per = kGradWaves / grad_shape(dim, k).w;
  const uint32_t need = (total + per - 1) / per;
  if (need == 0) return 0;
  const uint64_t bytes = static_cast<uint64_t>(total) * (k == Kind::kF32 ? 4 : 2);
  const uint32_t most = bytes >= kManyRowBytes ? kNormGradGrid : kNormGradGrid / 2;
  const uint32_t turns = (need + most - 1) / most;
  return (need + turns - 1) / turns;
}

hipError_t launch_norm(const NormArgs& a, Kind k, hipStream_t s) {
  if (a.total == 0) return hipSuccess;
  const Shape sh = forward_shape(a.dim, k);
  switch (k) {
    case Kind::kF32: return run_norm<EF32>(a, sh, s);
    case Kind::kBF16: return run_norm<EBF16>(a, sh, s);
    default: return run_norm<EF16>(a, sh, s);
  }
}

hipError_t launch_norm_grad(const NormGradArgs& a, Kind k, hipStream_t s) {
  const uint32_t grid = norm_grad_grid(a.total, a.dim, k);
  if (grid == 0) return hipSuccess;
  const Shape sh = grad_shape(a.dim, k);
  switch (k) {
    case Kind::kF32: return run_norm_grad<EF32>(a, sh, grid, s);
    case Kind::kBF16: return run_norm_grad<EBF16>(a, sh, grid, s);
    default: return run_norm_grad<EF16>(a, sh, grid, s);
  }
}

hipError_t launch_norm_join(const NormJoinArgs& a, Kind k, hipStream_t s) {
  const uint32_t sides = (a.dweight ? 1 : 0) + (a.dbias ? 1 : 0);
  if (sides == 0) return hipSuccess;
  const dim3 g((a.dim + 15) / 16, sides);
  switch (k) {
    case Kind::kF32: hipLaunchKernelGGL(k_norm_join<EF32>, g, dim3(256), 0, s, a); break;
    case Kind::kBF16: hipLaunchKernelGGL(k_norm_join<EBF16>, g, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL(k_norm_join<EF16>, g, dim3(256), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace rr
