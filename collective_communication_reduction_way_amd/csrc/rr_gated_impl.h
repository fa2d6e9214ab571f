// rr_gated_impl.h -- the matrix products of the gated column-parallel
// projections on the matrix cores (gfx950), one element kind per translation
// unit.
//
//   A = X Wg^T, U = X Wu^T, H = act(A) U;
//   dX = dA Wg + dU Wu;  dWg = dA^T X, dWu = dU^T X.
//
// The tile routine is rr_mfma.h's.  Forward, a tile's M axis alternates 16 rows of
// the gate with the same 16 rows of up, so that a lane holds both products of a
// feature and token and the activation costs no exchange and no memory.
//
// What bounds them.  Many tokens: the matrix cores and the power they take.  8192
// tokens, dim 4096, 16384 features, bfloat16: forward 1.82-1.95 ms with both products kept
// in float32 (1170 TFLOP/s, 2.4 GB leave), dhidden 1.59 (1380 TFLOP/s), the weights'
// gradients 1.60 (1370); the matrix cores are busy 60, 75 and 78 % of the cycles at 1.7 to
// 1.85 GHz.  A large library product reaches 1370.  Few tokens: the weights' read.  Between
// them: first loads and outputs, which only another workgroup of the unit overlaps.
#pragma once

#include <type_traits>

#include "rr_device.h"
#include "rr_gated_device.h"
#include "rr_mfma.h"
#include "rr_rows.h"

namespace rr {

// KC over pairs: 32 rows are 16 of the gate and the same 16 of up, of one shard;
// one load of a wavefront, of which 0 and 1 read the gate and 2 and 3 up.
template <int R>
struct KcPairLoader {
  static constexpr int NQ = R / 32;
  uint32_t off[1];
  Span m[NQ];
  RowWalk w;
  uint32_t mine;

  __device__ __forceinline__ void init(const GatedShards& sh, uint64_t stride, uint32_t f0, uint32_t f_end,
                                       uint32_t kbytes, int wave, int lane) {
    static_assert(kWaves == 4, "two wavefronts a weight");
    mine = wave * 1024;
    const uint32_t chunk = kc_chunk(wave * 8 + (lane >> 3), lane & 7) * 16;
    off[0] = ((wave & 1) * 8 + (lane >> 3)) * static_cast<uint32_t>(stride) + chunk;
    int r = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint32_t f = f0 + q * 16;
      m[q].set(nullptr, 0);
      if (f < f_end) {
        r = shard_of(sh, f, r);
        const uint32_t local = f - sh.off[r];
        const uint32_t n = local < sh.rows[r] ? (sh.rows[r] - local < 16 ? sh.rows[r] - local : 16) : 0;
        if (n)
          m[q].set(static_cast<const char*>(wave < 2 ? sh.gate[r] : sh.up[r]) + local * stride,
                   n * static_cast<uint32_t>(stride));
      }
    }
    w.init(kbytes, chunk, 0, (kbytes + 127) / 128);
    w.start(off, m);
  }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void load(int q, uint32_t lds) {
    load_to_lds(m[q], off[0], lds + mine, q * kWaves * 1024);
  }
  __device__ __forceinline__ void advance() { w.advance(off, m); }
};

// KS over the columns [c, end) of both weights, in runs of kFeat: a step's rows
// are rows of one shard of one weight, rows past its end read zeros.
template <class E, int R>
struct KsPairLoader {
  static constexpr int NQ = KsOffsets<E, R>::NQ;
  KsOffsets<E, R> o;
  const GatedShards* sh;
  uint64_t stride;
  uint32_t col0;     // bytes, as `cols`
  Span m;            // the next step's rows, at the tile's first column
  uint64_t gate;     // the run's first row of each weight, at the tile's first column
  uint64_t up;
  uint32_t rows;     // rows of the shard from there on
  uint32_t c, end;   // column of the next step; of the end
  uint32_t turn;     // where the next shard starts
  int r;
  uint32_t mine;

  __device__ __forceinline__ void init(const GatedShards& sh_, uint64_t stride_, uint32_t col0_, uint64_t cols,
                                       uint32_t c_, uint32_t end_, int wave, int lane) {
    mine = wave * 1024;
    sh = &sh_;
    stride = stride_;
    col0 = __builtin_amdgcn_readfirstlane(col0_);
    c = __builtin_amdgcn_readfirstlane(c_);
    end = __builtin_amdgcn_readfirstlane(end_);
    r = -1;
    turn = 0;
    rows = 0;
    gate = up = 0;
    m.set(nullptr, 0);
    fix(m);
    o.init(static_cast<uint32_t>(stride), cols, wave, lane);
  }
  __device__ __forceinline__ void place() {
    const uint32_t k = c % kFeat;  // rows of the run before this step
    const uint32_t have = rows > k ? rows - k : 0;
    const uint32_t n = have < Frag<E>::kBK ? have : Frag<E>::kBK;
    const uint64_t base = (c & kFeat ? up : gate) + k * stride;
    m.r[0] = static_cast<uint32_t>(base);
    m.r[1] = static_cast<uint32_t>(base >> 32);
    m.r[2] = __builtin_amdgcn_readfirstlane(
        n && c < end ? n * static_cast<uint32_t>(stride) - col0 : 0);
    fix(m);
  }
  // Before a step: the shard that holds it.
  __device__ __forceinline__ void prepare() {
    if (c >= turn && c < end) {
      do ++r;
      while (c >= 2 * sh->off[r + 1]);  // c < 2 off[p]: ends at the shard that holds c
      const uint32_t local = (c - 2 * sh->off[r]) / (2 * kFeat) * kFeat;
      turn = __builtin_amdgcn_readfirstlane(2 * sh->off[r + 1]);
      rows = __builtin_amdgcn_readfirstlane(sh->rows[r] > local ? sh->rows[r] - local : 0);
      gate = reinterpret_cast<uint64_t>(uniform(static_cast<const char*>(sh->gate[r]) + local * stride + col0));
      up = reinterpret_cast<uint64_t>(uniform(static_cast<const char*>(sh->up[r]) + local * stride + col0));
      place();
    }
  }
  __device__ __forceinline__ void load(int q, uint32_t lds) {
    load_to_lds(m, o.off[q], lds + mine, q * kWaves * 1024);
  }
  __device__ __forceinline__ void advance() {
    c += Frag<E>::kBK;
    if (c % (2 * kFeat) == 0) {
      gate += kFeat * stride;
      up += kFeat * stride;
      rows = __builtin_amdgcn_readfirstlane(rows < kFeat ? 0 : rows - kFeat);
    }
    place();
  }
};

// ---------------------------------------------------------------------------
// Forward: M = pairs of features, N = tokens, K = dim.  2048 x 4096 x 11008 bfloat16 in 256
// x 256 tiles 315 us (1170 TFLOP/s, three rounds of tiles over the chip where 2.7 are
// full); the products again with their gradients (kGrad), 1500 x 1024 x 4096: 42-46 us,
// 16 steps and an output of three matrices.

// Where the values of padded features f .. of token 0 are: which = 0: h (or dh),
// 1: A, 2: U (or their gradients).
struct GatedRow {
  char* base;       // NULL: nowhere
  uint64_t stride;  // bytes between tokens
  uint32_t n;       // features from f on
  bool vec;         // rows are 16-byte aligned
};
template <uint32_t ESZ>
__device__ __forceinline__ GatedRow gated_row(const GatedArgs& a, int which, uint32_t f) {
  GatedRow o{nullptr, 0, 0, true};
  if (f >= a.f1) return o;
  if (which > 0 && a.pre) {
    o.n = kFeat - f % kFeat;  // the run's padding is written too
    o.base = static_cast<char*>(a.pre) + (gate_col(f) + (which - 1) * kFeat) * ESZ;
    o.stride = a.pre_ld * ESZ;
    return o;
  }
  const int r = shard_of(a.sh, f);
  const uint32_t local = f - a.sh.off[r];
  o.n = local < a.sh.rows[r] ? a.sh.rows[r] - local : 0;
  char* const p = static_cast<char*>(which == 0 ? a.h[r] : which == 1 ? a.a[r] : a.u[r]);
  o.base = p + local * ESZ;
  o.stride = static_cast<uint64_t>(a.sh.rows[r]) * ESZ;
  o.vec = ((reinterpret_cast<uintptr_t>(p) | o.stride) & 15) == 0;
  return o;
}

// Four values, rounded to the kind's type.
template <class E>
__device__ __forceinline__ void put_four(char* to, const float* v) {
  if constexpr (sizeof(typename E::S) == 4) {
    *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[0], v[1], v[2], v[3]};
  } else if constexpr (__is_same(E, EBF16)) {
    *reinterpret_cast<uint2*>(to) = make_uint2(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]));
  } else {
    *reinterpret_cast<uint2*>(to) = make_uint2(f32x2_to_f16x2_bits(v[0], v[1]), f32x2_to_f16x2_bits(v[2], v[3]));
  }
}

// LDS rows of a tile's values: a token's BM / 2 features and 16 bytes.
template <class T, uint32_t ESZ>
constexpr uint32_t kPairRow = T::BM / 2 * ESZ + 16;

// A tile in LDS to or from memory, 16 bytes a lane along the rows.
template <class EO, class T, bool STORE>
__device__ __forceinline__ void move_tile(const GatedArgs& a, int which, uint32_t fbase, uint32_t t0, char* lds) {
  using S = typename EO::S;
  constexpr uint32_t V = kEpc<EO>, kRow = kPairRow<T, sizeof(S)>;
  constexpr uint32_t kChunks = T::BM / 2 / V, kRows = kWaves * 64 / kChunks;
  const uint32_t c = threadIdx.x % kChunks, row0 = threadIdx.x / kChunks;
  const GatedRow o = gated_row<sizeof(S)>(a, which, fbase + c * V);
  if (STORE && o.n == 0) return;
#pragma unroll 8
  for (uint32_t i = row0; i < T::BN; i += kRows) {
    const uint32_t t = t0 + i;
    u32x4* const q = reinterpret_cast<u32x4*>(lds + i * kRow + c * 16);
    S* const p = reinterpret_cast<S*>(o.base + t * o.stride);
    if constexpr (STORE) {
      if (t >= a.tokens) break;
      // (nontemporal: what leaves is read behind the other tiles' outputs; 8192 x 4096 x
      // 16384 step 5.51 -> 5.46 ms)
      if (o.vec && o.n >= V) __builtin_nontemporal_store(*q, reinterpret_cast<u32x4*>(p));
      else store_chunk<EO>(p, 0, o.n, *q);
    } else {
      *q = t < a.tokens ? load_chunk<EO>(p, 0, o.n) : u32x4{0, 0, 0, 0};
    }
  }
}

template <class E, class T, GatedAct ACT, GatedMode MODE>
__global__ __launch_bounds__(kWaves * 64) void k_gated(GatedArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  using S = typename E::S;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t tm, tn;
  tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t fbase = a.f0 + tm * (T::BM / 2), t0 = tn * T::BN;

  KcPairLoader<T::BM> la;
  KcLoader<T::BN> lb;
  const uint32_t steps = (a.kbytes + 127) / 128;
  // (all tiles start at their rows' beginning: starts spread along the rows, which
  // help where a pass over the weights bounds, cost 2 to 4 % here)
  la.init(a.sh, a.w_stride, fbase, a.f1, a.kbytes, wave, lane);
  lb.init(a.x, a.x_stride, t0, a.tokens, a.kbytes, 0, steps, wave, lane);
  k_start<T>(lds, la, lb);
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, steps, acc, la, lb,
      [&](uint32_t t, int m, int s) { return frag_kc<E>(t, m0, m, s, lane); },
      [&](uint32_t t, int n, int s) { return frag_kc<E>(t, n0, n, s, lane); });

  // Registers 4i + j and 8 + 4i + j of fragment m: gate and up of the tile's feature
  // m0 / 2 + 16 m + 8 i + 4 (lane / 32) + j, i < 2.  The values pass through LDS, a
  // matrix at a time, and leave in rows.
  const int half = (lane >> 5) * 4;
  const auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < T::NT; ++n)
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) f(acc[m][n], 4 * i, n0 + n * 32 + (lane & 31), m0 / 2 + m * 16 + i * 8 + half);
  };
  const auto put = [&](auto eo, char* to, uint32_t row, uint32_t col, const float* v) __attribute__((always_inline)) {
    using EO = decltype(eo);
    put_four<EO>(to + row * kPairRow<T, sizeof(typename EO::S)> + col * sizeof(typename EO::S), v);
  };
  if constexpr (MODE == GatedMode::kForward) {
    // which = 0: h, 1: A, 2: U; eo: the kind they are kept in
    const auto emit = [&](auto w, auto eo) __attribute__((always_inline)) {
      constexpr int which = decltype(w)::value;
      using EO = decltype(eo);
      static_assert(T::BN * kPairRow<T, sizeof(typename EO::S)> <= T::LDS, "the tile fits");
      __syncthreads();
      each([&](const f32x16_t& c, int x, uint32_t row, uint32_t col) __attribute__((always_inline)) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = which == 0 ? activate<E, ACT, false>(c[x + j], nullptr) * c[8 + x + j]
                            : which == 1 ? c[x + j] : c[8 + x + j];
        put(eo, lds, row, col, v);
      });
      __syncthreads();
      move_tile<EO, T, true>(a, which, fbase, t0, lds);
    };
    if (a.has_pre) {
      if (sizeof(S) == 2 && a.pre32) {
        emit(std::integral_constant<int, 1>{}, EF32{});
        emit(std::integral_constant<int, 2>{}, EF32{});
      } else {
        emit(std::integral_constant<int, 1>{}, E{});
        emit(std::integral_constant<int, 2>{}, E{});
      }
    }
    if (a.has_h) emit(std::integral_constant<int, 0>{}, E{});
  } else {
    // the gradients take the place of the products, side by side with dh where both fit
    constexpr uint32_t kTile = T::BN * kPairRow<T, sizeof(S)>;
    char* const to = lds + (2 * kTile <= T::LDS ? kTile : 0);
    move_tile<E, T, false>(a, 0, fbase, t0, lds);
    __syncthreads();
    each([&](f32x16_t& c, int x, uint32_t row, uint32_t col) __attribute__((always_inline)) {
      const S* const q = reinterpret_cast<const S*>(lds + row * kPairRow<T, sizeof(S)>) + col;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float da = c[x + j], du = c[8 + x + j];
        gate_grad_one<E, ACT>(load_one<E>(q + j), da, du);
        c[x + j] = da;
        c[8 + x + j] = du;
      }
    });
#pragma unroll
    for (int which = 1; which < 3; ++which) {
      if (which == 2 || 2 * kTile > T::LDS) __syncthreads();
      each([&](const f32x16_t& c, int x, uint32_t row, uint32_t col) __attribute__((always_inline)) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = which == 1 ? c[x + j] : c[8 + x + j];
        put(E{}, to, row, col, v);
      });
      __syncthreads();
      move_tile<E, T, true>(a, which, fbase, t0, to);
    }
  }
}

// ---------------------------------------------------------------------------
// Forward for few tokens: one pass over the weights at the rate of the memory.
// A workgroup takes 16 features, gate in rows 0 .. 15 of a 32-row product and up
// in rows 16 .. 31, and its four wavefronts share K, a step of 128 bytes a row in
// turn.  Each stages its own steps: loads of whole 128-byte lines at any
// alignment into registers, D steps ahead, from there into LDS of its own, so
// that no barrier holds the loads up.  No load of the loop is conditional: what a
// branch may skip the compiler has to wait for at once (24 x 2048 x 5504: 16.4 us with
// branches at any D, 14.8 without; 128 x 4096 x 11008 124 and 74).  The four sums are added in
// order.  One token at 4096 x 11008: 29.6 us, 180 MB at 6.1 TB/s; 24 at 2048 x 5504: 14.1
// us, 45 MB at 3.2 TB/s, most of it launch, first loads and the sums' way out.
//   X8: groups of 8 token rows.
template <int X8>
constexpr uint32_t kFewStage = (32 + (X8 + 3) / 4 * 32) * 128;  // bytes of LDS a wavefront

template <class E, int X8, int D, GatedAct ACT, GatedMode MODE>
__global__ __launch_bounds__(kWaves * 64) void k_gated_few(GatedArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[kWaves * kFewStage<X8>];
  using S = typename E::S;
  constexpr uint32_t V = 16 / sizeof(S), BK = Frag<E>::kBK;
  constexpr int NT = (X8 + 3) / 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t f0 = a.f0 + blockIdx.x * 16, t0 = blockIdx.y * (8 * X8);
  const int r = shard_of(a.sh, f0);
  const uint32_t local = f0 - a.sh.off[r];
  const uint32_t have = local < a.sh.rows[r] ? a.sh.rows[r] - local : 0;
  const uint32_t feats = have < 16 ? have : 16;
  const uint32_t tokens = a.tokens - t0 < 8 * X8 ? a.tokens - t0 : 8 * X8;
  if (feats == 0) {
    if (a.pre)  // columns that pad a run are zeros
      for (uint32_t i = threadIdx.x; i < tokens * 32; i += kWaves * 64) {
        const uint64_t at = (t0 + i / 32) * a.pre_ld + gate_col(f0 + i % 16) + (i & 16 ? kFeat : 0);
        if (a.pre32) static_cast<float*>(a.pre)[at] = 0.f;
        else static_cast<S*>(a.pre)[at] = S(0);
      }
    return;
  }

  // Load q of the weights: rows 8q .. 8q+7 of the product; of x: tokens 8q .. 8q+7.
  // Rows and tokens that do not exist repeat the last one that does; their results
  // are not stored.
  const uint32_t lr = lane >> 3, lc = lane & 7;
  const S* row[4 + X8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t f = (q & 1) * 8 + lr, n = local + (f < feats ? f : feats - 1);
    row[q] = static_cast<const S*>(q < 2 ? a.sh.gate[r] : a.sh.up[r]) + static_cast<uint64_t>(n) * a.dim;
  }
#pragma unroll
  for (int q = 0; q < X8; ++q) {
    const uint32_t t = q * 8 + lr < tokens ? q * 8 + lr : tokens - 1;
    row[4 + q] = static_cast<const S*>(a.x) + static_cast<uint64_t>(t0 + t) * a.dim;
  }
  char* const mine = lds + wave * kFewStage<X8>;

  f32x16_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x16_t{};
  // this wavefront's LDS: nothing but the order of its own accesses is needed
  const auto product = [&](const u32x4 (&v)[4 + X8]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4 + X8; ++q)
      *reinterpret_cast<u32x4*>(mine + (q * 8 + lr) * 128 + kc_chunk(q * 8 + lr, lc) * 16) = v[q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Frag<E> w = frag_kc<E>(lds_at(mine), 0, 0, s, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n] = mma<E>(w, frag_kc<E>(lds_at(mine) + 4096, 0, n, s, lane), acc[n]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  // Steps without a row's end: wave, wave + 4, ...
  const uint32_t whole = a.dim / BK;
  const uint32_t mine_steps = whole > static_cast<uint32_t>(wave) ? (whole - wave + kWaves - 1) / kWaves : 0;
  if (mine_steps > 0) {
    // Workgroups start at different places of their rows: rows are often a power of two
    // apart, and with every workgroup at the same place the chip would read from a few
    // memory channels at a time (one token at 4096 x 11008 33.1 -> 30.4 us).
    const uint32_t turn = blockIdx.x * 2 % whole;
    u32x4 v[D][4 + X8];
    const auto fetch = [&](int d, uint32_t i) __attribute__((always_inline)) {
      uint32_t k = wave + (i < mine_steps ? i : mine_steps - 1) * kWaves + turn;  // past the end: the last one, unused
      k -= k < whole ? 0 : whole;
      const uint32_t e = k * BK + lc * V;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[d][q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row[q] + e));
#pragma unroll
      for (int q = 4; q < 4 + X8; ++q) v[d][q] = *reinterpret_cast<const u32x4_any*>(row[q] + e);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, d);
    for (uint32_t i = 0; i < mine_steps; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (D > 1 && i + d >= mine_steps) {  // a turn that is not whole: weights of zero
#pragma unroll
          for (int q = 0; q < 4; ++q) v[d][q] = u32x4{0, 0, 0, 0};
          // (and tokens: what they hold may be infinite)
#pragma unroll
          for (int q = 4; q < 4 + X8; ++q) v[d][q] = u32x4{0, 0, 0, 0};
        }
        product(v[d]);
        fetch(d, i + d + D);
      }
    }
  }
  // the step with the row's end
  if (a.dim % BK && wave == static_cast<int>(whole % kWaves)) {
    u32x4 v[4 + X8];
#pragma unroll
    for (int q = 0; q < 4 + X8; ++q) v[q] = load_chunk<E>(row[q], whole * BK + lc * V, a.dim);
    product(v);
  }

  // [wave][token][32 rows and 4]
  constexpr uint32_t kRow = 36;
  float* const sum = reinterpret_cast<float*>(lds);
  static_assert(kWaves * 32 * NT * kRow * 4 <= kWaves * kFewStage<X8>, "the sums fit");
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4_t*>(sum + ((wave * NT + n) * 32 + (lane & 31)) * kRow + 8 * i + (lane >> 5) * 4) =
          f32x4_t{acc[n][4 * i], acc[n][4 * i + 1], acc[n][4 * i + 2], acc[n][4 * i + 3]};
  __syncthreads();
  const uint32_t f = threadIdx.x % 16;
  if (f >= feats && !a.pre) return;
  constexpr uint32_t esz = sizeof(S);
  const GatedRow oh = gated_row<esz>(a, 0, f0 + f);
  const GatedRow oa = a.pre32 ? gated_row<4>(a, 1, f0 + f) : gated_row<esz>(a, 1, f0 + f);
  const GatedRow ou = a.pre32 ? gated_row<4>(a, 2, f0 + f) : gated_row<esz>(a, 2, f0 + f);
  for (uint32_t t = threadIdx.x / 16; t < tokens; t += kWaves * 4) {
    float g = 0.f, u = 0.f;
    const uint64_t at = t0 + t;
    if (f < feats) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* const q = sum + (w * NT * 32 + t) * kRow;
        g += q[f];
        u += q[16 + f];
      }
      if constexpr (MODE == GatedMode::kGrad)
        gate_grad_one<E, ACT>(load_one<E>(reinterpret_cast<const S*>(oh.base + at * oh.stride)), g, u);
      else if (a.has_h)
        store_one<E>(reinterpret_cast<S*>(oh.base + at * oh.stride), activate<E, ACT, false>(g, nullptr) * u);
    }
    if (a.has_pre) {
      char* const qa = oa.base + at * oa.stride;
      char* const qu = ou.base + at * ou.stride;
      if (a.pre32) {
        *reinterpret_cast<float*>(qa) = g;
        *reinterpret_cast<float*>(qu) = u;
      } else {
        store_one<E>(reinterpret_cast<S*>(qa), g);
        store_one<E>(reinterpret_cast<S*>(qu), u);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The gradients' way out: the tile as rows of M in LDS, from there 16 bytes a lane
// along the rows, at any alignment.  (Written from the accumulators, where a lane holds
// four values of a row, an instruction touches 32 rows or, with odd rows, 64 places: 333 x
// 770 x 2050 dhidden and its activation 57 -> 49 us, weights the same 44 -> 38, in bfloat16
// 37 -> 28 and 24 -> 15.5.)  A tile that does not fit goes in two halves of each wavefront's
// rows.
//   factor(n): what row n is multiplied with; slot(n): where the run of up to 64 rows
//   from n on goes; cols: values of a row that exist.
template <class E, class T>
constexpr uint32_t kOutRow = T::BM * sizeof(typename E::S) + 16;

template <class E, class T, class F, class SLOT>
__device__ __forceinline__ void leave(char* lds, const f32x16_t (&acc)[T::MT][T::NT], int wave, int lane, uint32_t cols,
                                      F factor, SLOT slot) {
  using S = typename E::S;
  constexpr int kParts = T::BN * kOutRow<E, T> <= T::LDS ? 1 : 2, NP = T::NT / kParts;
  constexpr uint32_t kPart = NP * 32, kRun = kPart * T::WN < 64 ? kPart * T::WN : 64;
  static_assert(kPart * T::WN * kOutRow<E, T> <= T::LDS, "the part fits");
  static_assert(kParts == 1 || kRun == kPart, "a run is one wavefront's");
  constexpr uint32_t V = kEpc<E>, kChunks = T::BM / V, kRows = kWaves * 64 / kChunks;
  const uint32_t wm = wave / T::WN, wn = wave % T::WN;
  const uint32_t c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
#pragma unroll
  for (int q = 0; q < kParts; ++q) {
    if (q > 0) __syncthreads();
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const float f = factor(wn * (T::NT * 32) + (q * NP + n) * 32 + (lane & 31));
      char* const row = lds + (wn * kPart + n * 32 + (lane & 31)) * kOutRow<E, T>;
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          char* const to = row + (wm * (T::MT * 32) + m * 32 + i * 8 + (lane >> 5) * 4) * sizeof(S);
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = acc[m][q * NP + n][4 * i + j] * f;
          put_four<E>(to, v);
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kPart * T::WN / kRun; ++i) {
      const OutRows o = slot(kParts == 1 ? i * kRun : i * (T::NT * 32) + q * kPart);
      u32x4 v[kRun / kRows];
#pragma unroll
      for (uint32_t j = 0; j < kRun / kRows; ++j)
        v[j] = *reinterpret_cast<const u32x4*>(lds + (i * kRun + r0 + j * kRows) * kOutRow<E, T> + c * 16);
#pragma unroll
      for (uint32_t j = 0; j < kRun / kRows; ++j)
        if (r0 + j * kRows < o.rows)
          store_chunk<E>(reinterpret_cast<S*>(o.base + (r0 + j * kRows) * o.stride), c * V, cols, v[j]);
    }
  }
}

// The same in float32 into rows of sums.
template <class T>
__device__ __forceinline__ void leave_sums(const f32x16_t (&acc)[T::MT][T::NT], float* out, uint32_t ld, uint32_t row0,
                                           uint32_t rows, uint32_t col0, uint32_t cols, int wave, int lane, bool add) {
  const uint32_t m0 = wave / T::WN * (T::MT * 32), n0 = wave % T::WN * (T::NT * 32);
#pragma unroll
  for (int n = 0; n < T::NT; ++n) {
    const uint32_t t = row0 + n0 + n * 32 + (lane & 31);
    if (t >= rows) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = col0 + m0 + m * 32 + i * 8 + (lane >> 5) * 4;
        if (d >= cols) continue;
        f32x4_t* const q = reinterpret_cast<f32x4_t*>(out + static_cast<uint64_t>(t) * ld + d);
        f32x4_t v = {acc[m][n][4 * i], acc[m][n][4 * i + 1], acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
        if (add) {
          const f32x4_t o = *q;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += o[j];
        }
        *q = v;
      }
  }
}

// ---------------------------------------------------------------------------
// dhidden: M = dim, N = tokens, K = the piece's columns, in `splits` parts.
// Where that is all of K the result is written, else float32 sums.  (Few tokens give
// few tiles and all features as K: 96 x 768 x 2048 float16 7.2 us in 42 parts, 1500 x 1024 x
// 4096 bfloat16 37 in 5 and 7 for their join.)
template <class E, class T>
__global__ __launch_bounds__(kWaves * 64) void k_gated_hidden(GatedHiddenArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  using S = typename E::S;
  constexpr int esz = sizeof(S);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t id = blockIdx.x;
  if constexpr (T::BN < 256) {
    if (id < a.riders) {
      // each wavefront copies its share of kGatedRiderRows rows
      int top = 0;
      if constexpr (__is_same(E, EF16)) {
        if (a.copy.row_exp) {
          top = top_exponent<kWaves * 64>(a.copy.row_exp, a.copy.tokens, reinterpret_cast<int*>(lds));
          if (id == 0 && threadIdx.x == 0) *a.copy.scale = top;
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < kGatedRiderRows / kWaves; ++i) {
        const uint32_t t = id * kGatedRiderRows + i * kWaves + wave;
        if (t < a.copy.tokens) copy_scaled<E, 64>(a.copy, t, lane, top);
      }
      return;
    }
    id -= a.riders;
  }
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  const uint32_t split = id / tiles;
  uint32_t tm, tn;
  tile_of(id % tiles, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t d0 = tm * T::BM, t0 = tn * T::BN;
  const uint32_t all = (a.c1 - a.c0) / Frag<E>::kBK;
  const uint32_t k_lo = static_cast<uint64_t>(all) * split / a.splits;
  const uint32_t k_hi = static_cast<uint64_t>(all) * (split + 1) / a.splits;

  KsPairLoader<E, T::BM> la;
  KcLoader<T::BN> lb;
  // (a part that starts inside a run of 64 columns has read nothing of it yet)
  la.init(a.sh, a.w_stride, d0 * esz, a.w_stride - static_cast<uint64_t>(d0) * esz,
          a.c0 + k_lo * Frag<E>::kBK, a.c0 + k_hi * Frag<E>::kBK, wave, lane);
  lb.init(a.grad, a.ld * esz, t0, a.tokens, (a.c1 - a.c0) * esz, k_lo, k_hi - k_lo, wave, lane);
  k_start<T>(lds, la, lb);
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, k_hi - k_lo, acc, la, lb,
      [&](uint32_t t, int m, int s) { return frag_ks<E, T::BM>(t, m0, m, s, lane); },
      [&](uint32_t t, int n, int s) { return frag_kc<E>(t, n0, n, s, lane); });
  if (a.out) {
    leave<E, T>(
        lds, acc, wave, lane, a.dim - d0,
        [&](uint32_t n) {
          if constexpr (__is_same(E, EF16)) {
            if (t0 + n < a.tokens) return ldexpf(1.f, -row_scale(a.row_max[t0 + n]));
          }
          return 1.f;
        },
        [&](uint32_t n) {
          const uint32_t t = t0 + n;
          return OutRows{reinterpret_cast<char*>(static_cast<S*>(a.out) + static_cast<uint64_t>(t) * a.dim + d0),
                         static_cast<uint64_t>(a.dim) * sizeof(S), t < a.tokens ? a.tokens - t : 0};
        });
    return;
  }
  leave_sums<T>(acc, a.acc + split * a.split_stride, a.acc_ld, t0, a.tokens, d0, a.dim, wave, lane, a.add);
}

// ---------------------------------------------------------------------------
// dgate and dup: M = dim, N = columns, K = tokens.  1500 x 1024 x 4096 29 us (870 TFLOP/s:
// 512 tiles of 128 x 128 with 24 steps each); 96 x 768 x 2048 float16 6.2 us, launch, first
// loads and output.
template <class E, class T>
__global__ __launch_bounds__(kWaves * 64) void k_gated_weight(GatedWeightArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  using S = typename E::S;
  constexpr int esz = sizeof(S);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t id = blockIdx.x;
  if constexpr (T::BN < 256) {
    const uint32_t i = id - a.rider0;
    if (i < a.riders) {
      const uint32_t t = i / a.join_cols, by = i % a.join_cols;
      float* const part = reinterpret_cast<float*>(lds);
      if (t >= a.tokens) return;
      if (a.join.splits >= kGatedJoinMany) join_sums<E, 4>(a.join, t, by, part);
      else join_sums<E, 1>(a.join, t, by, part);
      return;
    }
    if (a.rider0 == 0) id -= a.riders;
  }
  const uint32_t tiles = a.tiles_m * a.tiles_n, split = id / tiles;
  uint32_t tm, tn;
  tile_of(id % tiles, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t d0 = tm * T::BM, v0 = a.c0 + tn * T::BN;
  const uint32_t all = (a.tokens + Frag<E>::kBK - 1) / Frag<E>::kBK;  // steps
  const uint32_t k_lo = static_cast<uint64_t>(all) * split / a.splits;
  const uint32_t k_hi = static_cast<uint64_t>(all) * (split + 1) / a.splits;
  const uint32_t first = k_lo * Frag<E>::kBK;
  const uint32_t last = k_hi * Frag<E>::kBK < a.tokens ? k_hi * Frag<E>::kBK : a.tokens;
  KsLoader<E, T::BM> la;
  KsLoader<E, T::BN> lb;
  la.init(static_cast<const char*>(a.x) + first * a.x_stride + static_cast<uint64_t>(d0) * esz, a.x_stride,
          a.x_stride - static_cast<uint64_t>(d0) * esz, last - first, wave, lane);
  lb.init(static_cast<const char*>(a.grad) + (first * a.ld + v0) * esz, a.ld * esz,
          static_cast<uint64_t>(a.c1 - v0) * esz, last - first, wave, lane);
  k_start<T>(lds, la, lb);
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, k_hi - k_lo, acc, la, lb,
      [&](uint32_t t, int m, int s) { return frag_ks<E, T::BM>(t, m0, m, s, lane); },
      [&](uint32_t t, int n, int s) { return frag_ks<E, T::BN>(t, n0, n, s, lane); });
  if constexpr (T::BN < 256) {
    if (a.splits > 1) {
      leave_sums<T>(acc, a.acc + split * a.acc_stride, a.acc_ld, v0, a.c1, d0, a.dim, wave, lane, false);
      return;
    }
  }
  float scale = 1.f;
  if constexpr (__is_same(E, EF16)) scale = ldexpf(1.f, a.scale[0] - 30);
  // The rows from column c on: a feature's row of one shard of one weight.
  const auto rows_at = [&](uint32_t n) {
    const uint32_t c = v0 + n;
    OutRows o{nullptr, static_cast<uint64_t>(a.dim) * sizeof(S), 0};
    if (c >= a.c1) return o;
    const uint32_t f = c / (2 * kFeat) * kFeat + c % kFeat;
    const int r = shard_of(a, f);
    const uint32_t local = f - a.off[r];
    o.rows = local < a.rows[r] ? a.rows[r] - local : 0;
    if (o.rows)
      o.base = static_cast<char*>(c & kFeat ? a.dup[r] : a.dgate[r]) +
               (static_cast<uint64_t>(local) * a.dim + d0) * sizeof(S);
    return o;
  };
  leave<E, T>(lds, acc, wave, lane, a.dim - d0, [&](uint32_t) { return scale; }, rows_at);
}

// ---------------------------------------------------------------------------
// gated_small of the kind
template <class E>
using GatedSmall = std::conditional_t<sizeof(typename E::S) == 4, T64, T128>;

template <class E, GatedAct ACT, GatedMode MODE>
hipError_t run_gated(const GatedArgs& a, GatedTile t, hipStream_t s) {
  const dim3 b(kWaves * 64);
  if (t == GatedTile::kFew) {
    const uint32_t x8 = (a.tokens + 7) / 8;
#define RR_FEW(X8, D)                                                                             \
    if (x8 <= X8 || X8 == 16) {                                                                   \
      const dim3 g((a.f1 - a.f0) / 16, (x8 + X8 - 1) / X8);                                       \
      hipLaunchKernelGGL((k_gated_few<E, X8, D, ACT, MODE>), g, b, 0, s, a);                      \
      return hipGetLastError();                                                                   \
    }
    RR_FEW(1, 2)
    RR_FEW(4, 2)
    RR_FEW(8, 2)
    RR_FEW(16, 1)
#undef RR_FEW
  }
  const dim3 g(a.tiles_m * a.tiles_n);
  if (t == GatedTile::k256x256) hipLaunchKernelGGL((k_gated<E, T256, ACT, MODE>), g, b, 0, s, a);
  else if (t == GatedTile::k64x64) hipLaunchKernelGGL((k_gated<E, T64x64, ACT, MODE>), g, b, 0, s, a);
  else if (sizeof(typename E::S) == 2 && t == GatedTile::k256x192)
    hipLaunchKernelGGL((k_gated<E, std::conditional_t<sizeof(typename E::S) == 2, T192, GatedSmall<E>>, ACT, MODE>), g,
                       b, 0, s, a);
  else hipLaunchKernelGGL((k_gated<E, GatedSmall<E>, ACT, MODE>), g, b, 0, s, a);
  return hipGetLastError();
}

// float16's gradients are scaled by their row: k_gate_grad_f16 forms them.
template <class E, GatedAct ACT>
hipError_t run_gated_mode(const GatedArgs& a, GatedMode m, GatedTile t, hipStream_t s) {
  if constexpr (!__is_same(E, EF16)) {
    if (m == GatedMode::kGrad) return run_gated<E, ACT, GatedMode::kGrad>(a, t, s);
  }
  return run_gated<E, ACT, GatedMode::kForward>(a, t, s);
}

template <class E>
hipError_t run_gated_hidden(const GatedHiddenArgs& a, GatedTile t, hipStream_t s) {
  const dim3 g(a.riders + a.tiles_m * a.tiles_n * a.splits), b(kWaves * 64);
  switch (t) {
    case GatedTile::k256x256: hipLaunchKernelGGL((k_gated_hidden<E, T256>), g, b, 0, s, a); break;
    case GatedTile::k128x32: hipLaunchKernelGGL((k_gated_hidden<E, T32>), g, b, 0, s, a); break;
    default: hipLaunchKernelGGL((k_gated_hidden<E, GatedSmall<E>>), g, b, 0, s, a); break;
  }
  return hipGetLastError();
}

template <class E>
hipError_t run_gated_weight(const GatedWeightArgs& a, GatedTile t, hipStream_t s) {
  const dim3 g(a.riders + a.tiles_m * a.tiles_n * a.splits), b(kWaves * 64);
  if (t == GatedTile::k256x256) hipLaunchKernelGGL((k_gated_weight<E, T256>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_gated_weight<E, GatedSmall<E>>), g, b, 0, s, a);
  return hipGetLastError();
}

#define RR_GATED_UNIT(NAME, E)                                                                               \
  hipError_t launch_gated_##NAME(const GatedArgs& a, GatedAct act, GatedMode m, GatedTile t, hipStream_t s) { \
    return act == GatedAct::kSilu ? run_gated_mode<E, GatedAct::kSilu>(a, m, t, s)                          \
                                  : run_gated_mode<E, GatedAct::kGelu>(a, m, t, s);                         \
  }                                                                                                         \
  hipError_t launch_gated_hidden_##NAME(const GatedHiddenArgs& a, GatedTile t, hipStream_t s) {   \
    return run_gated_hidden<E>(a, t, s);                                                          \
  }                                                                                               \
  hipError_t launch_gated_weight_##NAME(const GatedWeightArgs& a, GatedTile t, hipStream_t s) {   \
    return run_gated_weight<E>(a, t, s);                                                          \
  }

}  // namespace rr
