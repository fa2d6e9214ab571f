// rr_vocab_impl.h -- the matrix products of the vocabulary-parallel softmax
// cross entropy on the matrix cores (gfx950), one element kind per translation
// unit.
//
//   z = X W^T;  forward: max and sum of exp over each tile of the vocabulary;
//   G = g (exp(z - lse) - onehot);  dX = G W;  dW = G^T X.
//
// One tile routine serves the three products: acc[m][n] = sum_k A(m,k) B(n,k)
// with a BM x BN tile in the accumulators of 4 or 8 wavefronts.  An operand
// is staged in LDS in the layout it has in memory:
//   KC: rows are the M (or N) axis and k runs along a row (128 bytes a step);
//   KS: rows are the k axis and M (or N) runs along a row.  16-bit fragments of
//       such a tile are read with the transposing LDS load, so neither the
//       weights nor the gradient of the logits are ever transposed in memory.
// Both layouts permute 16-byte chunks within a row by an XOR of row bits, so
// that the fragment reads hit all 64 banks; the permutation is applied to the
// global address, because the direct global-to-LDS load writes its 64 x 16
// bytes consecutively.
#pragma once

#include "rr_device.h"
#include "rr_vocab_device.h"

namespace rr {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

#define RR_LDS __attribute__((address_space(3)))
#define RR_GLB __attribute__((address_space(1)))

// What out-of-range chunks read.
static __device__ __attribute__((aligned(16))) uint32_t vocab_zero[4];

// 16 bytes a lane from memory straight into LDS; `lds` is the wavefront's base
// and lane l's chunk lands at lds + 16 l.
__device__ __forceinline__ void load_to_lds(const void* g, char* lds) {
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const RR_GLB void*>(reinterpret_cast<uintptr_t>(g)),
                                   reinterpret_cast<RR_LDS void*>(static_cast<uint32_t>(
                                       reinterpret_cast<uintptr_t>(lds))),
                                   16, 0, 0);
}

template <class E>
struct Frag {
  static constexpr int kEsz = static_cast<int>(sizeof(typename E::S));
  static constexpr int kBK = 128 / kEsz;  // k per step
  static constexpr int kEPC = 16 / kEsz;  // elements per 16-byte chunk
  u32x4 v;
};

// One step of a 16 x 16 product: 32 values of k in 16-bit types, 16 in float32
// (there lane group g holds k = 4g .. 4g+3, and the j-th instruction multiplies
// the four values k = 4g + j).
template <class E>
__device__ __forceinline__ f32x4_t mma(const Frag<E>& a, const Frag<E>& b, f32x4_t c) {
  if constexpr (__is_same(E, EBF16)) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                   __builtin_bit_cast(bf16x8_t, b.v), c, 0, 0, 0);
  } else if constexpr (__is_same(E, EF16)) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a.v),
                                                  __builtin_bit_cast(f16x8_t, b.v), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[j]), __uint_as_float(b.v[j]), c, 0, 0, 0);
    return c;
  }
}

// ---------------------------------------------------------------------------
// LDS layouts.

// KS: the permutation of a row's units of 16 elements.  16-bit: lanes 0-31 of
// a transposing read touch rows 8g + (0..3), g = 0, 1, of one unit.  float32: a
// read touches rows 4g, g = 0..3, of one unit.
template <class E>
__device__ __forceinline__ uint32_t ks_swizzle(uint32_t k) {
  if constexpr (sizeof(typename E::S) == 2) {
    return (k & 3u) | ((k >> 1) & 4u);
  } else {
    return (k >> 2) & 3u;
  }
}

// Fragment of rows r0 .. r0+15 of a KC tile, k substep s (0 or 1).
template <class E>
__device__ __forceinline__ Frag<E> frag_kc(const char* tile, int r0, int s, int lane) {
  const int row = r0 + (lane & 15);
  const int chunk = (s * 4 + (lane >> 4)) ^ (lane & 7);
  Frag<E> f;
  f.v = *reinterpret_cast<const u32x4*>(tile + row * 128 + chunk * 16);
  return f;
}

// Fragment of columns c0 .. c0+15 of a KS tile of R columns.
template <class E, int R>
__device__ __forceinline__ Frag<E> frag_ks(const char* tile, int c0, int s, int lane) {
  Frag<E> f;
  if constexpr (sizeof(typename E::S) == 2) {
    const int k = s * 32 + (lane >> 4) * 8 + ((lane >> 2) & 3);
    const uint32_t unit = static_cast<uint32_t>(c0 >> 4) ^ ks_swizzle<E>(k);
    const char* q = tile + k * (R * 2) + unit * 32 + (lane & 3) * 8;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<RR_LDS s16x4_t*>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q))));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<RR_LDS s16x4_t*>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q + 4 * R * 2))));
    const s16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    f.v = __builtin_bit_cast(u32x4, v);
  } else {
    const int k = s * 16 + (lane >> 4) * 4;
    const uint32_t unit = static_cast<uint32_t>(c0 >> 4) ^ ks_swizzle<E>(k);
    const char* q = tile + k * (R * 4) + unit * 64 + (lane & 15) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = *reinterpret_cast<const uint32_t*>(q + j * (R * 4));
  }
  return f;
}

// The global 16-byte chunk that belongs at LDS chunk `pos` of a row.
__device__ __forceinline__ uint32_t kc_chunk(uint32_t row, uint32_t pos) { return pos ^ (row & 7u); }
template <class E>
__device__ __forceinline__ uint32_t ks_chunk(uint32_t k, uint32_t pos) {
  if constexpr (sizeof(typename E::S) == 2) {
    return (((pos >> 1) ^ ks_swizzle<E>(k)) << 1) | (pos & 1u);
  } else {
    return (((pos >> 2) ^ ks_swizzle<E>(k)) << 2) | (pos & 3u);
  }
}

// ---------------------------------------------------------------------------
// Loaders.  A tile of R rows or columns is R*128 bytes = R/8 wavefront loads;
// wavefront w of NW issues loads w, w + NW, ...

// KC: row pointers fixed for the whole product; k advances 128 bytes a step.
template <int R, int NW>
struct KcLoader {
  static constexpr int NQ = R / 8 / NW;
  const char* ptr[NQ];   // row + this lane's chunk, or the zero chunk
  uint32_t left;         // bytes of the row from the lane's chunk on (0 for a row out of range: see step)
  uint32_t in_row;       // bit q: row q is in range
  uint32_t base;         // LDS offset of the wavefront's first load

  template <class ROW>
  __device__ __forceinline__ void init(ROW row_ptr, uint32_t kbytes, int wave, int lane) {
    in_row = 0;
    const uint32_t chunk = kc_chunk(lane >> 3, lane & 7);
    left = kbytes > chunk * 16 ? kbytes - chunk * 16 : 0;
    base = wave * 1024;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const char* r = row_ptr((wave + q * NW) * 8 + (lane >> 3));
      if (r) {
        ptr[q] = r + chunk * 16;
        in_row |= 1u << q;
      } else {
        ptr[q] = reinterpret_cast<const char*>(vocab_zero);
      }
    }
  }
  // Skip to k step kt.
  __device__ __forceinline__ void seek(uint32_t kt) {
    const uint32_t b = kt * 128;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (in_row >> q & 1) ptr[q] += b;
    left = left > b ? left - b : 0;
  }
  // Issue the loads of the next step.
  __device__ __forceinline__ void step(char* lds) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const char* g = left ? ptr[q] : reinterpret_cast<const char*>(vocab_zero);
      load_to_lds(g, lds + base + q * NW * 1024);
      if (in_row >> q & 1) ptr[q] += 128;
    }
    left = left > 128 ? left - 128 : 0;
  }
};

// KS with rows at a constant stride: row k of step kt is base + (kt*BK + k)*stride.
// `cols` is the number of valid bytes of a row from the tile's first column on.
template <class E, int R, int NW>
struct KsLoader {
  static constexpr int NQ = R / 8 / NW;
  static constexpr int RB = R * static_cast<int>(sizeof(typename E::S));
  const char* ptr[NQ];
  uint64_t step_bytes;
  uint32_t in_cols;
  uint32_t base;

  __device__ __forceinline__ void init(const void* src, uint64_t stride, uint64_t cols, uint32_t kt, int wave,
                                       int lane) {
    step_bytes = stride * Frag<E>::kBK;
    in_cols = 0;
    base = wave * 1024;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint32_t o = (wave + q * NW) * 1024 + lane * 16;
      const uint32_t k = o / RB;
      const uint32_t c = ks_chunk<E>(k, (o % RB) / 16) * 16;
      if (c < cols) {
        ptr[q] = static_cast<const char*>(src) + kt * step_bytes + k * stride + c;
        in_cols |= 1u << q;
      } else {
        ptr[q] = reinterpret_cast<const char*>(vocab_zero);
      }
    }
  }
  __device__ __forceinline__ void step(char* lds) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      load_to_lds(ptr[q], lds + base + q * NW * 1024);
      if (in_cols >> q & 1) ptr[q] += step_bytes;
    }
  }
};

// KS over the padded vocabulary: a step's rows are rows of one shard, rows
// past its end read zeros.
template <class E, int R, int NW>
struct KsShardLoader {
  static constexpr int NQ = R / 8 / NW;
  static constexpr int RB = R * static_cast<int>(sizeof(typename E::S));
  uint64_t rel[NQ];      // byte offset of the lane's chunk from the step's first row and the tile's first column
  uint32_t krow[NQ];
  uint32_t in_cols;
  uint32_t base;
  uint64_t stride;
  uint64_t col0;
  uint32_t c;            // padded column of the next step
  int r;                 // its shard

  __device__ __forceinline__ void init(const VocabShards& sh, uint64_t stride_, uint64_t col0_, uint64_t cols,
                                       uint32_t c_, int wave, int lane) {
    in_cols = 0;
    base = wave * 1024;
    stride = stride_;
    col0 = col0_;
    c = c_;
    r = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint32_t o = (wave + q * NW) * 1024 + lane * 16;
      const uint32_t k = o / RB;
      const uint32_t cc = ks_chunk<E>(k, (o % RB) / 16) * 16;
      krow[q] = k;
      rel[q] = k * stride + cc;
      if (cc < cols) in_cols |= 1u << q;
    }
  }
  __device__ __forceinline__ void step(const VocabShards& sh, char* lds) {
    while (c >= sh.off[r + 1]) ++r;  // c < off[p]: ends at the shard that holds c
    const uint32_t local = c - sh.off[r];
    // rows of the shard from this step on (none in a slot's padded second half)
    const uint32_t rows = sh.rows[r] > local ? sh.rows[r] - local : 0;
    const char* b = static_cast<const char*>(sh.w[r]) + local * stride + col0;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const bool in = (in_cols >> q & 1) && krow[q] < rows;
      load_to_lds(in ? b + rel[q] : reinterpret_cast<const char*>(vocab_zero), lds + base + q * NW * 1024);
    }
    c += Frag<E>::kBK;
  }
};

// ---------------------------------------------------------------------------
// Tile configurations: BM x BN in WM x WN wavefronts.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int ABYTES = BM * 128, BBYTES = BN * 128;
  static constexpr int STAGE = ABYTES + BBYTES;
};
using T256 = Tile<256, 256, 2, 4>;
using T128 = Tile<128, 128, 2, 2>;
using T32 = Tile<128, 32, 4, 1>;

// The K loop: two LDS stages, the loads of step k+1 in flight while step k is
// multiplied.  `issue(lds)` issues the loads of the next step, `fa(tile, m, s)`
// and `fb(tile, n, s)` read fragments.
template <class E, class T, class ISSUE, class FA, class FB>
__device__ __forceinline__ void k_loop(char* lds, uint32_t steps, f32x4_t (&acc)[T::MT][T::NT], ISSUE issue, FA fa,
                                       FB fb) {
#pragma unroll
  for (int m = 0; m < T::MT; ++m)
#pragma unroll
    for (int n = 0; n < T::NT; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (steps == 0) return;
  issue(lds);
  __syncthreads();  // waits for the loads as well
  for (uint32_t k = 0; k < steps; ++k) {
    char* cur = lds + (k & 1) * T::STAGE;
    if (k + 1 < steps) issue(lds + ((k + 1) & 1) * T::STAGE);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Frag<E> a[T::MT], b[T::NT];
#pragma unroll
      for (int n = 0; n < T::NT; ++n) b[n] = fb(cur + T::ABYTES, n, s);
#pragma unroll
      for (int m = 0; m < T::MT; ++m) a[m] = fa(cur, m, s);
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int n = 0; n < T::NT; ++n) acc[m][n] = mma<E>(a[m], b[n], acc[m][n]);
    }
    __syncthreads();
  }
}

// Workgroup -> tile.  Consecutive workgroups go to the 8 XCDs in turn, so each
// XCD is given a contiguous run of the tile order, and that order walks
// blocks of 8 M tiles by all N tiles, so that the workgroups an XCD runs at
// one time share operand panels in its L2.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tm, uint32_t tn, uint32_t& m, uint32_t& n) {
  const uint32_t total = tm * tn;
  const uint32_t per = total / 8, rem = total % 8, x = id % 8;
  const uint32_t i = x * per + (x < rem ? x : rem) + id / 8;
  const uint32_t g = i / (8 * tn);
  const uint32_t width = tm - g * 8 < 8 ? tm - g * 8 : 8;
  const uint32_t j = i - g * 8 * tn;
  m = g * 8 + j % width;
  n = j / width;
}

// ---------------------------------------------------------------------------
// Logits: M = vocabulary, N = tokens.  A lane of an accumulator holds 4
// consecutive columns of one token.
template <class E, class T, bool GRAD>
__global__ __launch_bounds__(T::NW * 64) void k_logits(LogitArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t tm, tn;
  tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t cbase = a.c0 + tm * T::BM;
  const uint32_t t0 = tn * T::BN;

  KcLoader<T::BM, T::NW> la;
  KcLoader<T::BN, T::NW> lb;
  la.init(
      [&](uint32_t row) -> const char* {
        const uint32_t c = cbase + row;
        const char* q = nullptr;
        for (int r = 0; r < a.sh.p; ++r)
          if (c >= a.sh.off[r] && c - a.sh.off[r] < a.sh.rows[r])
            q = static_cast<const char*>(a.sh.w[r]) + static_cast<uint64_t>(c - a.sh.off[r]) * a.w_stride;
        return c < a.c1 ? q : nullptr;
      },
      a.kbytes, wave, lane);
  lb.init(
      [&](uint32_t row) -> const char* {
        const uint32_t t = t0 + row;
        return t < a.tokens ? static_cast<const char*>(a.x) + t * a.x_stride : nullptr;
      },
      a.kbytes, wave, lane);
  f32x4_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 16), n0 = wn * (T::NT * 16);
  k_loop<E, T>(
      lds, (a.kbytes + 127) / 128, acc,
      [&](char* l) {
        la.step(l);
        lb.step(l + T::ABYTES);
      },
      [&](const char* t, int m, int s) { return frag_kc<E>(t, m0 + m * 16, s, lane); },
      [&](const char* t, int n, int s) { return frag_kc<E>(t, n0 + n * 16, s, lane); });

  // Which of this lane's 4 columns per M fragment exist: bit 4m + j.
  const uint32_t lc = cbase + m0 + (lane >> 4) * 4;
  uint32_t have = 0;
  for (int r = 0; r < a.sh.p; ++r) {
    const uint32_t lo = a.sh.off[r], hi = lo + a.sh.rows[r];
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = lc + m * 16 + j;
        if (c >= lo && c < hi && c < a.c1) have |= 1u << (4 * m + j);
      }
  }

  if constexpr (!GRAD) {
    float* red = reinterpret_cast<float*>(lds);  // [WM][BN][2]
#pragma unroll
    for (int n = 0; n < T::NT; ++n) {
      const uint32_t t = t0 + n0 + n * 16 + (lane & 15);
      float mx = -__builtin_inff();
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!(have >> (4 * m + j) & 1)) acc[m][n][j] = -__builtin_inff();
          mx = fmaxf(mx, acc[m][n][j]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      // a tile whose logits are all -inf has sum 0, not NaN
      const float ref = mx == -__builtin_inff() ? 0.f : mx;
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += __expf(acc[m][n][j] - ref);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (lane < 16) {
        float* q = red + (wm * T::BN + n0 + n * 16 + lane) * 2;
        q[0] = mx;
        q[1] = sum;
      }
      if (t < a.tokens) {
        const uint32_t col = padded_col(a.sh, target_at(a.targets, a.target_bytes, t));
#pragma unroll
        for (int m = 0; m < T::MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col == lc + m * 16 + j && (have >> (4 * m + j) & 1)) a.hit[t] = acc[m][n][j];
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < T::BN; i += T::NW * 64) {
      const uint32_t t = t0 + i;
      if (t >= a.tokens) continue;
      float mx = red[i * 2], sum = red[i * 2 + 1];
#pragma unroll
      for (int w = 1; w < T::WM; ++w) {
        const float m2 = red[(w * T::BN + i) * 2], s2 = red[(w * T::BN + i) * 2 + 1];
        const float top = fmaxf(mx, m2);
        const float ref = top == -__builtin_inff() ? 0.f : top;
        sum = sum * __expf(mx - ref) + s2 * __expf(m2 - ref);
        mx = top;
      }
      float* q = a.part + (static_cast<uint64_t>(a.tile0 + tm) * a.tokens + t) * 2;
      q[0] = mx;
      q[1] = sum;
    }
  } else {
    using S = typename E::S;
#pragma unroll
    for (int n = 0; n < T::NT; ++n) {
      const uint32_t t = t0 + n0 + n * 16 + (lane & 15);
      if (t >= a.grad_rows) continue;
      uint32_t col = kMasked;
      float lse = 0.f, g = 0.f;
      if (t < a.tokens) {
        col = a.tcol[t];
        lse = a.lse[t];
        g = a.grad_loss[t];
      }
      const bool live = col != kMasked;
      if constexpr (__is_same(E, EF16)) g = ldexpf(g, 15 - token_exponent(g));
      S* out = static_cast<S*>(a.grad) + t * a.ld;
#pragma unroll
      for (int m = 0; m < T::MT; ++m) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pr = __expf(acc[m][n][j] - lse) - (col == lc + m * 16 + j ? 1.f : 0.f);
          v[j] = live && (have >> (4 * m + j) & 1) ? pr * g : 0.f;
        }
        const uint32_t c = lc + m * 16 - a.c0;
        if constexpr (sizeof(S) == 2) {
          // The target's entry is the row's largest by far; what its rounding
          // takes goes into the two products on the side (k_join,
          // k_weight_grad), which leaves the rounding of the outputs the
          // largest error.
          const uint32_t j = col - (lc + m * 16);
          if (live && j < 4) {
            const float x = j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3];
            a.lo[t] = x - half_to_f32<E>(f32_to_half<E>(x));
          }
        }
        if (c < a.c1 - a.c0) {
          if constexpr (sizeof(S) == 4) {
            *reinterpret_cast<f32x4_t*>(out + c) = f32x4_t{v[0], v[1], v[2], v[3]};
          } else {
            uint32_t w0, w1;
            if constexpr (__is_same(E, EBF16)) {
              w0 = f32x2_to_bf16x2_bits(v[0], v[1]);
              w1 = f32x2_to_bf16x2_bits(v[2], v[3]);
            } else {
              w0 = f32x2_to_f16x2_bits(v[0], v[1]);
              w1 = f32x2_to_f16x2_bits(v[2], v[3]);
            }
            *reinterpret_cast<uint2*>(out + c) = make_uint2(w0, w1);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// dhidden: M = dim, N = tokens, K = the piece's padded columns, in `splits`
// parts.  Accumulated in float32.
template <class E, class T>
__global__ __launch_bounds__(T::NW * 64) void k_hidden_grad(HiddenGradArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[2 * T::STAGE];
  constexpr int esz = sizeof(typename E::S);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  const uint32_t split = blockIdx.x / tiles;
  uint32_t tm, tn;
  tile_of(blockIdx.x % tiles, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t d0 = tm * T::BM, t0 = tn * T::BN;
  const uint32_t all = (a.c1 - a.c0) / Frag<E>::kBK;
  const uint32_t k_lo = static_cast<uint64_t>(all) * split / a.splits;
  const uint32_t k_hi = static_cast<uint64_t>(all) * (split + 1) / a.splits;

  KsShardLoader<E, T::BM, T::NW> la;
  KcLoader<T::BN, T::NW> lb;
  la.init(a.sh, a.w_stride, static_cast<uint64_t>(d0) * esz, static_cast<uint64_t>(a.dim - d0) * esz,
          a.c0 + k_lo * Frag<E>::kBK, wave, lane);
  lb.init(
      [&](uint32_t row) -> const char* {
        const uint32_t t = t0 + row;
        return t < a.grad_rows ? static_cast<const char*>(a.grad) + t * a.ld * esz : nullptr;
      },
      (a.c1 - a.c0) * esz, wave, lane);
  lb.seek(k_lo);
  f32x4_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 16), n0 = wn * (T::NT * 16);
  k_loop<E, T>(
      lds, k_hi - k_lo, acc,
      [&](char* l) {
        la.step(a.sh, l);
        lb.step(l + T::ABYTES);
      },
      [&](const char* t, int m, int s) { return frag_ks<E, T::BM>(t, m0 + m * 16, s, lane); },
      [&](const char* t, int n, int s) { return frag_kc<E>(t, n0 + n * 16, s, lane); });
  float* out = a.acc + split * a.split_stride;
#pragma unroll
  for (int n = 0; n < T::NT; ++n) {
    const uint32_t t = t0 + n0 + n * 16 + (lane & 15);
    if (t >= a.tokens) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
      const uint32_t d = d0 + m0 + m * 16 + (lane >> 4) * 4;
      float* q = out + static_cast<uint64_t>(t) * a.dim + d;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (d + j < a.dim) q[j] = a.add ? q[j] + acc[m][n][j] : acc[m][n][j];
    }
  }
}

// ---------------------------------------------------------------------------
// dweights: M = dim, N = the piece's padded columns, K = tokens.
template <class E, class T>
__global__ __launch_bounds__(T::NW * 64) void k_weight_grad(WeightGradArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[2 * T::STAGE];
  using S = typename E::S;
  constexpr int esz = sizeof(S);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t tm, tn;
  tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t d0 = tm * T::BM, v0 = tn * T::BN;
  KsLoader<E, T::BM, T::NW> la;
  KsLoader<E, T::BN, T::NW> lb;
  la.init(static_cast<const char*>(a.xg) + static_cast<uint64_t>(d0) * esz, a.xg_stride,
          a.xg_stride - static_cast<uint64_t>(d0) * esz, 0, wave, lane);
  lb.init(static_cast<const char*>(a.grad) + static_cast<uint64_t>(v0) * esz, a.ld * esz,
          static_cast<uint64_t>(a.c1 - a.c0 - v0) * esz, 0, wave, lane);
  f32x4_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 16), n0 = wn * (T::NT * 16);
  k_loop<E, T>(
      lds, a.rows / Frag<E>::kBK, acc,
      [&](char* l) {
        la.step(l);
        lb.step(l + T::ABYTES);
      },
      [&](const char* t, int m, int s) { return frag_ks<E, T::BM>(t, m0 + m * 16, s, lane); },
      [&](const char* t, int n, int s) { return frag_ks<E, T::BN>(t, n0 + n * 16, s, lane); });
  if constexpr (esz == 2) {
    // What rounding took from the targets' entries: the tokens whose target
    // lies in this tile (few: the whole vocabulary shares the tokens) are
    // listed in order and added as further K steps of 64.
    __shared__ uint32_t list[64 + T::NW * 64];
    __shared__ uint32_t found[T::NW];
    const uint32_t first = a.c0 + v0;
    uint32_t have = 0;
    const auto add = [&](uint32_t n) {
#pragma unroll
      for (int q = 0; q < KsLoader<E, T::BM, T::NW>::NQ; ++q) {
        const uint32_t o = (wave + q * T::NW) * 1024 + lane * 16;
        const uint32_t k = o / (T::BM * esz);
        const uint32_t c = ks_chunk<E>(k, (o % (T::BM * esz)) / 16) * 16;
        const bool in = k < n && c < a.xg_stride - static_cast<uint64_t>(d0) * esz;
        load_to_lds(in ? static_cast<const char*>(a.xg) + list[k] * a.xg_stride + static_cast<uint64_t>(d0) * esz + c
                       : reinterpret_cast<const char*>(vocab_zero),
                    lds + o - lane * 16);
      }
      for (uint32_t i = threadIdx.x; i < T::BBYTES / 16; i += T::NW * 64)
        *reinterpret_cast<u32x4*>(lds + T::ABYTES + i * 16) = u32x4{0, 0, 0, 0};
      __syncthreads();
      if (threadIdx.x < n) {
        const uint32_t k = threadIdx.x, t = list[k], c = a.tcol[t] - first;
        const uint32_t at = k * (T::BN * esz) + (((c >> 4) ^ ks_swizzle<E>(k)) << 5) + (c & 15u) * 2;
        *reinterpret_cast<S*>(lds + T::ABYTES + at) = static_cast<S>(f32_to_half<E>(a.lo[t]));
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<E> fa[T::MT], fb[T::NT];
#pragma unroll
        for (int m = 0; m < T::MT; ++m) fa[m] = frag_ks<E, T::BM>(lds, m0 + m * 16, s, lane);
#pragma unroll
        for (int n2 = 0; n2 < T::NT; ++n2) fb[n2] = frag_ks<E, T::BN>(lds + T::ABYTES, n0 + n2 * 16, s, lane);
#pragma unroll
        for (int m = 0; m < T::MT; ++m)
#pragma unroll
          for (int n2 = 0; n2 < T::NT; ++n2) acc[m][n2] = mma<E>(fa[m], fb[n2], acc[m][n2]);
      }
      __syncthreads();
    };
    for (uint32_t b = 0; b < a.tokens; b += T::NW * 64) {
      const uint32_t t = b + threadIdx.x;
      const bool in = t < a.tokens && a.tcol[t] - first < T::BN;  // kMasked - first is out of range
      const uint64_t mask = __ballot(in);
      if (lane == 0) found[wave] = __popcll(mask);
      __syncthreads();
      uint32_t at = have, total = have;
#pragma unroll
      for (int w = 0; w < T::NW; ++w) {
        if (w < wave) at += found[w];
        total += found[w];
      }
      if (in) list[at + __popcll(mask & ((1ull << lane) - 1))] = t;
      have = total;
      __syncthreads();
      while (have >= 64) {
        add(64);
        const uint32_t left = have - 64;  // at most NW * 64 - 1
        const uint32_t v = threadIdx.x < left ? list[64 + threadIdx.x] : 0;
        __syncthreads();
        if (threadIdx.x < left) list[threadIdx.x] = v;
        __syncthreads();
        have = left;
      }
    }
    if (have > 0) add(have);
  }
  float scale = 1.f;
  if constexpr (__is_same(E, EF16)) scale = ldexpf(1.f, a.scale[0] - 15);
#pragma unroll
  for (int n = 0; n < T::NT; ++n) {
    const uint32_t c = a.c0 + v0 + n0 + n * 16 + (lane & 15);
    S* row = nullptr;
    if (c < a.c1)
      for (int r = 0; r < a.sh.p; ++r)
        if (c >= a.sh.off[r] && c - a.sh.off[r] < a.sh.rows[r])
          row = static_cast<S*>(a.dw[r]) + static_cast<uint64_t>(c - a.sh.off[r]) * a.dim;
    if (!row) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
      const uint32_t d = d0 + m0 + m * 16 + (lane >> 4) * 4;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = acc[m][n][j] * scale;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (d + j < a.dim) store_one<E>(row + d + j, v[j]);
    }
  }
}

// ---------------------------------------------------------------------------
template <class E>
hipError_t run_logits(const LogitArgs& a, VocabTile t, bool grad, hipStream_t s) {
  const dim3 g(a.tiles_m * a.tiles_n);
  if (g.x == 0) return hipSuccess;
#define RR_LAUNCH(TT)                                                        \
  if (grad)                                                                  \
    hipLaunchKernelGGL((k_logits<E, TT, true>), g, dim3(TT::NW * 64), 0, s, a); \
  else                                                                       \
    hipLaunchKernelGGL((k_logits<E, TT, false>), g, dim3(TT::NW * 64), 0, s, a);
  switch (t) {
    case VocabTile::k256x256: RR_LAUNCH(T256) break;
    case VocabTile::k128x128: RR_LAUNCH(T128) break;
    default: RR_LAUNCH(T32) break;
  }
#undef RR_LAUNCH
  return hipGetLastError();
}

template <class E>
hipError_t run_hidden_grad(const HiddenGradArgs& a, VocabTile t, hipStream_t s) {
  const dim3 g(a.tiles_m * a.tiles_n * a.splits);
  if (g.x == 0) return hipSuccess;
  switch (t) {
    case VocabTile::k256x256: hipLaunchKernelGGL((k_hidden_grad<E, T256>), g, dim3(T256::NW * 64), 0, s, a); break;
    case VocabTile::k128x128: hipLaunchKernelGGL((k_hidden_grad<E, T128>), g, dim3(T128::NW * 64), 0, s, a); break;
    default: hipLaunchKernelGGL((k_hidden_grad<E, T32>), g, dim3(T32::NW * 64), 0, s, a); break;
  }
  return hipGetLastError();
}

template <class E>
hipError_t run_weight_grad(const WeightGradArgs& a, VocabTile t, hipStream_t s) {
  const dim3 g(a.tiles_m * a.tiles_n);
  if (g.x == 0) return hipSuccess;
  if (t == VocabTile::k256x256)
    hipLaunchKernelGGL((k_weight_grad<E, T256>), g, dim3(T256::NW * 64), 0, s, a);
  else
    hipLaunchKernelGGL((k_weight_grad<E, T128>), g, dim3(T128::NW * 64), 0, s, a);
  return hipGetLastError();
}

#define RR_VOCAB_UNIT(NAME, E)                                                                 \
  hipError_t launch_logits_##NAME(const LogitArgs& a, VocabTile t, bool grad, hipStream_t s) { \
    return run_logits<E>(a, t, grad, s);                                                       \
  }                                                                                            \
  hipError_t launch_hidden_grad_##NAME(const HiddenGradArgs& a, VocabTile t, hipStream_t s) {  \
    return run_hidden_grad<E>(a, t, s);                                                        \
  }                                                                                            \
  hipError_t launch_weight_grad_##NAME(const WeightGradArgs& a, VocabTile t, hipStream_t s) {  \
    return run_weight_grad<E>(a, t, s);                                                        \
  }

}  // namespace rr
