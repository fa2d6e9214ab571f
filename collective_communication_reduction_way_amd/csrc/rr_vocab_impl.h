// rr_vocab_impl.h -- the matrix products of the vocabulary-parallel softmax
// cross entropy on the matrix cores (gfx950), one element kind per translation
// unit.
//
//   z = X W^T;  forward: max and sum of exp over each tile of the vocabulary;
//   G = g (exp(z - lse) - onehot);  dX = G W;  dW = G^T X.
//
// One tile routine serves the three products: acc[m][n] = sum_k A(m,k) B(n,k)
// with a BM x BN tile in the accumulators of 4 wavefronts.  An operand is
// staged in LDS in the layout it has in memory:
//   KC: rows are the M (or N) axis and k runs along a row (128 bytes a step);
//   KS: rows are the k axis and M (or N) runs along a row.  16-bit fragments of
//       such a tile are read with the transposing LDS load, so neither the
//       weights nor the gradient of the logits are ever transposed in memory.
// Both layouts permute 16-byte chunks within a row by an XOR of row bits, so
// that the fragment reads hit all 64 banks (no conflicts counted); the
// permutation is applied to the global address, because the direct
// global-to-LDS load writes its 64 x 16 bytes consecutively.
//
// What bounds the products.  The large tile: the matrix cores and the power
// they take.  8192 tokens, dim 4096, 50257 rows, bfloat16: logits 2.92 ms (1160
// TFLOP/s), their gradient 2.88, dhidden 2.58 (1310 TFLOP/s), dweights 2.77 in two
// launches; the matrix cores are busy 56-71% of the cycles at clocks of 1.55 to 1.75
// GHz (2.4 without load), and a loop of nothing but the products reaches 1590
// TFLOP/s on the same data.  A large library product reaches 1360.  A 256 x 256 tile on 4
// wavefronts (128 x 128 each) needs two thirds of the LDS reads of 8 wavefronts
// of 128 x 64, and 32 x 32 instructions keep its 256 accumulators in place where
// the compiler moved those of 16 x 16 ones about.  The small tiles: loads, and
// the first loads and the output, which nothing overlaps but the other
// workgroup of the compute unit.
#pragma once

#include <type_traits>

#include "rr_device.h"
#include "rr_vocab_device.h"

namespace rr {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

#define RR_LDS __attribute__((address_space(3)))
#define RR_GLB __attribute__((address_space(1)))

// A stretch of memory that a wavefront loads from: reads at or past `bytes` give
// zeros, which is how rows and columns that do not exist are read.
struct Span {
  const char* base;  // the same in every lane
  uint32_t bytes;
};
constexpr uint32_t kNoOffset = 0xFFFFFFF0u;  // past the end of every span

__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// 16 bytes a lane from memory straight into LDS; `lds` is the wavefront's base
// and lane l's chunk lands at lds + 16 l.  The instruction is written out
// because for the builtin the compiler waits for all loads in flight before the
// next transposing LDS read, whatever it reads.  Nothing comes back in
// registers; wait_for_loads() stands before the barrier after which the LDS is
// read.  (One wait state is due between the write of M0 and its use.)
__device__ __forceinline__ void load_to_lds(const Span& m, uint32_t offset, char* lds) {
  const uint64_t base = reinterpret_cast<uint64_t>(uniform(m.base));
  const u32x4 r = {static_cast<uint32_t>(base), static_cast<uint32_t>(base >> 32) & 0xFFFFu,
                   static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(m.bytes)), 0x00027000u};
  const uint32_t to = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((RR_LDS char*)lds)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is reserved: nothing of the compiler's lives in it
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset), "s"(r)
               : "m0");
#pragma clang diagnostic pop
}
__device__ __forceinline__ void wait_for_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <class E>
struct Frag {
  static constexpr int kEsz = static_cast<int>(sizeof(typename E::S));
  static constexpr int kBK = 128 / kEsz;  // k per step
  static constexpr int kEPC = 16 / kEsz;  // elements per 16-byte chunk
  u32x4 v;
};

// A 32 x 32 product over a quarter of a step: 16 values of k in 16-bit types (lane
// half h holds k = 8h .. 8h+7), 8 in float32 (half h holds k = 4h .. 4h+3, and the
// j-th instruction multiplies k = j and 4 + j).  Lane l of the result holds column
// l mod 32 and, in register 4i + j, row 8i + 4 (l / 32) + j.
template <class E>
__device__ __forceinline__ f32x16_t mma(const Frag<E>& a, const Frag<E>& b, f32x16_t c) {
  if constexpr (__is_same(E, EBF16)) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                   __builtin_bit_cast(bf16x8_t, b.v), c, 0, 0, 0);
  } else if constexpr (__is_same(E, EF16)) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a.v),
                                                  __builtin_bit_cast(f16x8_t, b.v), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.v[j]), __uint_as_float(b.v[j]), c, 0, 0, 0);
    return c;
  }
}

// ---------------------------------------------------------------------------
// LDS layouts.

// KS: the permutation of a row's units of 16 elements, chosen so that the rows
// and units that half a wavefront reads at once lie in different banks:
// 16-bit, rows k .. k+3 of two adjacent units (32 bytes each); float32, rows k
// and k+4 of two adjacent units (64 bytes each).
template <class E>
__device__ __forceinline__ uint32_t ks_swizzle(uint32_t k) {
  if constexpr (sizeof(typename E::S) == 2) {
    return (k & 3u) << 1;
  } else {
    return (k >> 1) & 2u;
  }
}

// Fragment of rows r0 .. r0+31 of a KC tile, quarter s of the step.
template <class E>
__device__ __forceinline__ Frag<E> frag_kc(const char* tile, int r0, int s, int lane) {
  const int row = r0 + (lane & 31);
  const int chunk = (s * 2 + (lane >> 5)) ^ ((lane >> 1) & 7);
  Frag<E> f;
  f.v = *reinterpret_cast<const u32x4*>(tile + row * 128 + chunk * 16);
  return f;
}

// Fragment of columns c0 .. c0+31 of a KS tile of R columns.
template <class E, int R>
__device__ __forceinline__ Frag<E> frag_ks(const char* tile, int c0, int s, int lane) {
  Frag<E> f;
  const uint32_t u = static_cast<uint32_t>(c0 >> 4) + ((lane >> 4) & 1);
  if constexpr (sizeof(typename E::S) == 2) {
    // 16 lanes read 4 rows of 16 columns and get a column of 4 rows each
    const int k = s * 16 + (lane >> 5) * 8 + ((lane >> 2) & 3);
    const char* q = tile + k * (R * 2) + (u ^ ks_swizzle<E>(k)) * 32 + (lane & 3) * 8;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (RR_LDS s16x4_t*)(q));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (RR_LDS s16x4_t*)(q + 4 * R * 2));
    const s16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    f.v = __builtin_bit_cast(u32x4, v);
  } else {
    const int k = s * 8 + (lane >> 5) * 4;
    const char* q = tile + k * (R * 4) + (u ^ ks_swizzle<E>(k)) * 64 + (lane & 15) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = *reinterpret_cast<const uint32_t*>(q + j * (R * 4));
  }
  return f;
}

// The global 16-byte chunk that belongs at LDS chunk `pos` of a row.
__device__ __forceinline__ uint32_t kc_chunk(uint32_t row, uint32_t pos) { return pos ^ ((row >> 1) & 7u); }
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
// wavefront w of the 4 issues loads w, w + 4, ...  Offsets within a tile are 32
// bits (a tile's 256 rows span less than 2^31 bytes), the bases advance.
constexpr int kWaves = 4;

// Where a KC operand stands in its rows: steps of 128 bytes from `first` on, round
// to the row's start and up to `first` again, `steps` in all.
struct RowWalk {
  uint32_t pos, end, steps;  // bytes; the row's bytes in whole steps; steps left
  __device__ __forceinline__ void init(uint32_t first, uint32_t steps_all, uint32_t steps_) {
    pos = first * 128;
    end = steps_all * 128;
    steps = steps_;
  }
  __device__ __forceinline__ void start(Span& m) const {
    m.base += pos;
    m.bytes = m.bytes && steps ? m.bytes - pos : 0;
  }
  // The bytes to the next step (negative round the end).
  __device__ __forceinline__ int32_t advance() {
    const bool wrap = pos + 128 == end;
    const int32_t d = wrap ? 128 - static_cast<int32_t>(end) : 128;
    pos += d;
    steps -= steps ? 1 : 0;
    return d;
  }
  // Nothing is read after the last step.
  __device__ __forceinline__ void move(Span& m, int32_t d) const {
    m.base += d;
    m.bytes = m.bytes && steps ? m.bytes - d : 0;
  }
};

// KC over rows at a constant stride: rows row0 .. of a matrix of `rows` rows.
template <int R>
struct KcLoader {
  static constexpr int NQ = R / 8 / kWaves;
  uint32_t off[NQ];
  uint32_t left;  // bytes of a row from the lane's chunk on
  Span m;
  RowWalk w;
  int wave;

  __device__ __forceinline__ void init(const void* src, uint64_t stride, uint32_t row0, uint32_t rows, uint32_t kbytes,
                                       uint32_t first, uint32_t steps, int wave_, int lane) {
    wave = wave_;
    const uint32_t chunk = kc_chunk(wave * 8 + (lane >> 3), lane & 7) * 16;
    left = kbytes > chunk ? kbytes - chunk : 0;
    const uint32_t n = row0 < rows ? (rows - row0 < R ? rows - row0 : R) : 0;
    m.base = uniform(static_cast<const char*>(src) + row0 * stride);
    m.bytes = n * static_cast<uint32_t>(stride);
    w.init(first, (kbytes + 127) / 128, steps);
    w.start(m);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      off[q] = ((wave + q * kWaves) * 8 + (lane >> 3)) * static_cast<uint32_t>(stride) + chunk;
  }
  __device__ __forceinline__ void prepare() {}
  // Load q of the next step (zeros after the last one).
  __device__ __forceinline__ void load(int q, char* lds) {
    load_to_lds(m, left > w.pos ? off[q] : kNoOffset, lds + (wave + q * kWaves) * 1024);
  }
  __device__ __forceinline__ void advance() { w.move(m, w.advance()); }
};

// KC over the padded vocabulary: a slot of kSlot columns is kSlot rows of one
// shard, and two of a wavefront's loads.
template <int R>
struct KcShardLoader {
  static constexpr int NS = R / kSlot, NQ = 2 * NS;
  static_assert(kSlot == 2 * 8 * kWaves, "two loads a slot");
  uint32_t off[2];
  uint32_t left;
  Span m[NS];
  RowWalk w;
  int wave;

  __device__ __forceinline__ void init(const VocabShards& sh, uint64_t stride, uint32_t col, uint32_t col_end,
                                       uint32_t kbytes, uint32_t first, int wave_, int lane) {
    wave = wave_;
    const uint32_t chunk = kc_chunk(wave * 8 + (lane >> 3), lane & 7) * 16;
    left = kbytes > chunk ? kbytes - chunk : 0;
    w.init(first, (kbytes + 127) / 128, (kbytes + 127) / 128);
#pragma unroll
    for (int i = 0; i < 2; ++i) off[i] = ((wave + i * kWaves) * 8 + (lane >> 3)) * static_cast<uint32_t>(stride) + chunk;
    int r = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint32_t c = col + s * kSlot;
      m[s] = Span{nullptr, 0};
      if (c < col_end) {
        while (c >= sh.off[r + 1]) ++r;  // c < off[p]: ends at the shard that holds c
        const uint32_t local = c - sh.off[r];
        const uint32_t n = sh.rows[r] - local < kSlot ? sh.rows[r] - local : kSlot;
        m[s].base = uniform(static_cast<const char*>(sh.w[r]) + local * stride);
        m[s].bytes = n * static_cast<uint32_t>(stride);
      }
      w.start(m[s]);
    }
  }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void load(int q, char* lds) {
    load_to_lds(m[q / 2], left > w.pos ? off[q % 2] : kNoOffset, lds + (wave + q * kWaves) * 1024);
  }
  __device__ __forceinline__ void advance() {
    const int32_t d = w.advance();
#pragma unroll
    for (int s = 0; s < NS; ++s) w.move(m[s], d);
  }
};

// Offsets of a KS tile's loads: `cols` valid bytes of a row from the tile's
// first column on.
template <class E, int R>
struct KsOffsets {
  static constexpr int NQ = R / 8 / kWaves;
  static constexpr int RB = R * static_cast<int>(sizeof(typename E::S));
  uint32_t off[NQ];
  __device__ __forceinline__ void init(uint32_t stride, uint64_t cols, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint32_t o = (wave + q * kWaves) * 1024 + lane * 16;
      const uint32_t k = o / RB;
      const uint32_t c = ks_chunk<E>(k, (o % RB) / 16) * 16;
      off[q] = c < cols ? k * stride + c : kNoOffset;
    }
  }
};

// KS with rows at a constant stride, all of them there.
template <class E, int R>
struct KsLoader {
  static constexpr int NQ = KsOffsets<E, R>::NQ;
  KsOffsets<E, R> o;
  Span m;
  uint64_t step_bytes;
  uint32_t steps;  // that are left
  int wave;

  __device__ __forceinline__ void init(const char* src, uint64_t stride, uint64_t cols, uint32_t steps_, int wave_,
                                       int lane) {
    wave = wave_;
    steps = steps_;
    o.init(static_cast<uint32_t>(stride), cols, wave, lane);
    step_bytes = stride * Frag<E>::kBK;
    m.base = uniform(src);
    // the step's rows, up to the last byte of the last one that belongs to the tile's columns
    m.bytes = static_cast<uint32_t>(step_bytes - stride + (cols < KsOffsets<E, R>::RB ? cols : KsOffsets<E, R>::RB));
  }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void load(int q, char* lds) {
    load_to_lds(Span{m.base, steps ? m.bytes : 0}, o.off[q], lds + (wave + q * kWaves) * 1024);
  }
  __device__ __forceinline__ void advance() {
    m.base += step_bytes;
    steps -= steps ? 1 : 0;
  }
};

// KS over the padded vocabulary, columns [c, end): a step's rows are rows of
// one shard, rows past its end read zeros.
template <class E, int R>
struct KsShardLoader {
  static constexpr int NQ = KsOffsets<E, R>::NQ;
  KsOffsets<E, R> o;
  const VocabShards* sh;
  uint64_t stride, col0;
  const char* base;  // the next step's first row, at the tile's first column
  uint32_t rows;     // rows of the shard from there on
  uint32_t c, end;   // padded column of the next step; of the end
  uint32_t turn;     // where the next shard starts
  int r;
  int wave;

  __device__ __forceinline__ void init(const VocabShards& sh_, uint64_t stride_, uint64_t col0_, uint64_t cols,
                                       uint32_t c_, uint32_t end_, int wave_, int lane) {
    wave = wave_;
    sh = &sh_;
    stride = stride_;
    col0 = col0_;
    c = c_;
    end = end_;
    r = -1;
    turn = 0;
    rows = 0;
    base = nullptr;
    o.init(static_cast<uint32_t>(stride), cols, wave, lane);
  }
  // Before a step: the shard that holds it.
  __device__ __forceinline__ void prepare() {
    if (c >= turn && c < end) {
      do ++r;
      while (c >= sh->off[r + 1]);  // c < off[p]: ends at the shard that holds c
      const uint32_t local = c - sh->off[r];
      turn = sh->off[r + 1];
      base = uniform(static_cast<const char*>(sh->w[r]) + local * stride + col0);
      rows = sh->rows[r] > local ? sh->rows[r] - local : 0;
    }
  }
  __device__ __forceinline__ void load(int q, char* lds) {
    const uint32_t n = rows < Frag<E>::kBK ? rows : Frag<E>::kBK;
    const Span m{base, n && c < end ? static_cast<uint32_t>(n * stride - col0) : 0};
    load_to_lds(m, o.off[q], lds + (wave + q * kWaves) * 1024);
  }
  __device__ __forceinline__ void advance() {
    c += Frag<E>::kBK;
    base += Frag<E>::kBK * stride;
    rows -= rows < Frag<E>::kBK ? rows : Frag<E>::kBK;
  }
};

// ---------------------------------------------------------------------------
// Tile configurations: BM x BN in WM x WN wavefronts.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static_assert(WM * WN == kWaves, "4 wavefronts");
  static constexpr int MT = BM / WM / 32, NT = BN / WN / 32;
  static constexpr int ABYTES = BM * 128, BBYTES = BN * 128;
  // LDS: three slots for A's tiles, two for B's (k_loop)
  static constexpr int LDS = 3 * ABYTES + 2 * BBYTES;
  static constexpr int BOFF = 3 * ABYTES;
};
using T256 = Tile<256, 256, 2, 2>;
using T128 = Tile<128, 128, 2, 2>;
// (float32: a compute unit's matrix cores are busy four times as long with the
// same bytes, so smaller tiles cost nothing and two of them fill each other's
// waits)
using T64 = Tile<128, 64, 2, 2>;
using T64x64 = Tile<64, 64, 2, 2>;
using T32 = Tile<128, 32, 4, 1>;

// The K loop.  A step is 128 bytes of k in four quarters.  While a quarter is
// multiplied the fragments of the next one are read; when those of the last
// quarter are there, everything in the step's tiles has been read, and the
// wavefronts meet, once a step.  A has three slots in LDS and B two: A's loads
// for the step after next go out during the first three quarters, into the free
// slot, B's during the last one, into the slot just read, so that the loads
// are spread over the step and have most of a step to arrive.
// `fa(tile, m, s)` and `fb(tile, n, s)` read the fragments of quarter s.
//
// The order within a quarter is the source's: left to itself the compiler reads
// the fragments where they are used and waits for each.
// A barrier that leaves memory loads in flight.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
template <int N>
__device__ __forceinline__ void wait_for_all_but() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The loads of the first two steps.
template <class T, class LA, class LB>
__device__ __forceinline__ void k_start(char* lds, LA& la, LB& lb) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    la.prepare();
#pragma unroll
    for (int q = 0; q < LA::NQ; ++q) la.load(q, lds + i * T::ABYTES);
#pragma unroll
    for (int q = 0; q < LB::NQ; ++q) lb.load(q, lds + T::BOFF + i * T::BBYTES);
    la.advance();
    lb.advance();
  }
}

// After k_start.  Until here the third slot of A, lds + 2 ABYTES, is free.
template <class E, class T, class LA, class LB, class FA, class FB>
__device__ __forceinline__ void k_loop(char* lds, uint32_t steps, f32x16_t (&acc)[T::MT][T::NT], LA& la, LB& lb, FA fa,
                                       FB fb) {
  constexpr int MT = T::MT, NT = T::NT, kMmas = MT * NT;
  // Where a wavefront has one product a quarter the quarters have four sums (64 x
  // 64 tiles: two, which leaves registers for four workgroups a compute unit):
  // shorter chains of roundings (one token, dim 768: logits off by up to 2e-6 at 12.7
  // with one sum, 9e-7 with four).
  constexpr int kMore = kMmas > 1 ? 0 : T::BM == 128 ? 3 : 1;
  f32x16_t more[kMore ? kMore : 1];
#pragma unroll
  for (int i = 0; i < kMore; ++i) more[i] = f32x16_t{};
  constexpr int kFirst = kMmas > 1 ? kMmas / 2 : 1;        // the products that the reads go between
  constexpr int kReads = (MT + NT + kFirst - 1) / kFirst;  // fragments read before each of them
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x16_t{};
  if (steps == 0) {  // (the loads of k_start read zeros)
    wait_for_loads();
    __syncthreads();
    return;
  }
  Frag<E> a[2][MT], b[2][NT];
  const auto read = [&](int to, int i, const char* ta, const char* tb, int s) __attribute__((always_inline)) {
    if (i < NT) b[to][i] = fb(tb, i, s);
    else if (i < NT + MT) a[to][i - NT] = fa(ta, i - NT, s);
  };
  char* const lds_b = lds + T::BOFF;
  wait_for_all_but<LA::NQ + LB::NQ>();
  meet();
#pragma unroll
  for (int i = 0; i < NT + MT; ++i) read(0, i, lds, lds_b, 0);
  uint32_t slot = 0;  // of A: k mod 3
  for (uint32_t k = 0; k < steps; ++k) {
    const uint32_t slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot == 0 ? 2 : slot - 1;
    const char* const ac = lds + slot * T::ABYTES;
    const char* const an = lds + slot1 * T::ABYTES;
    char* const af = lds + slot2 * T::ABYTES;
    char* const bc = lds_b + (k & 1) * T::BBYTES;
    const char* const bn = lds_b + (~k & 1) * T::BBYTES;
    slot = slot1;
    la.prepare();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 3) {
        wait_for_all_but<LA::NQ>();
        meet();
      }
#pragma unroll
      for (int i = 0; i < kMmas; ++i) {
#pragma unroll
        for (int j = i * kReads; j < (i + 1) * kReads; ++j) {
          if (s < 3) read(~s & 1, j, ac, bc, s + 1);
          else read(0, j, an, bn, 0);  // after the last step: what lies there, unused
        }
        // loads past the last step read zeros, unused
        if (s < 3) {
          constexpr int kAll = 3 * kMmas;
          const int at = s * kMmas + i;
#pragma unroll
          for (int q = at * LA::NQ / kAll; q < (at + 1) * LA::NQ / kAll; ++q) la.load(q, af);
        } else {
#pragma unroll
          for (int q = i * LB::NQ / kMmas; q < (i + 1) * LB::NQ / kMmas; ++q) lb.load(q, bc);
        }
        constexpr int kSums = kMore + 1;
        f32x16_t& sum = s % kSums > 0 ? more[s % kSums > 0 ? s % kSums - 1 : 0] : acc[i / NT][i % NT];
        sum = mma<E>(a[s & 1][i / NT], b[s & 1][i % NT], sum);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    la.advance();
    lb.advance();
  }
  // The accumulators end the loop where they were in it (without this the
  // register allocator moved them about within it for the sake of what follows).
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) asm volatile("" : "+a"(acc[m][n]));
#pragma unroll
  for (int i = 0; i < kMore; ++i) asm volatile("" : "+a"(more[i]));
  if constexpr (kMore > 0) {
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      acc[0][0][x] += more[0][x];
      if constexpr (kMore == 3) acc[0][0][x] += more[1][x] + more[2][x];
    }
  }
  wait_for_loads();
  __syncthreads();  // the caller may use the LDS
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
// 16-bit results on their way out.  A lane of the accumulators holds 4
// consecutive values of M for one N, 8 bytes: written as they are, every
// instruction would touch 32 rows of the output for 16 bytes each.  They are laid
// down in LDS as rows of M instead (16 bytes of padding keep neighbouring rows
// in different banks), and leave as 16 bytes a lane along the rows.
template <class T>
constexpr uint32_t kRow16 = T::BM * 2 + 16;

template <class E, class T>
__device__ __forceinline__ void put16(char* lds, uint32_t n, uint32_t m, const float* v, uint32_t mask) {
  static_assert(T::BN * kRow16<T> <= T::LDS, "the tile fits");
  uint32_t w0, w1;
  if constexpr (__is_same(E, EBF16)) {
    w0 = f32x2_to_bf16x2_bits(v[0], v[1]);
    w1 = f32x2_to_bf16x2_bits(v[2], v[3]);
  } else {
    w0 = f32x2_to_f16x2_bits(v[0], v[1]);
    w1 = f32x2_to_f16x2_bits(v[2], v[3]);
  }
  *reinterpret_cast<uint2*>(lds + n * kRow16<T> + m * 2) = make_uint2(w0 & mask, w1 & mask);
}

// Rows of the tile in runs of up to 64: slot(i) says where run i goes (`rows` of
// them exist); `cols` values of a row exist, a multiple of 8.
struct OutRows {
  char* base;
  uint64_t stride;  // bytes
  uint32_t rows;
};
template <class E, class T, class SLOT>
__device__ __forceinline__ void take16(const char* lds, uint32_t cols, SLOT slot) {
  constexpr uint32_t kChunks = T::BM / 8, kRows = kWaves * 64 / kChunks, kRun = T::BN < 64 ? T::BN : 64;
  const uint32_t c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
#pragma unroll
  for (uint32_t i = 0; i < T::BN / kRun; ++i) {
    const OutRows o = slot(i);
    const uint32_t rows = c * 8 < cols ? o.rows : 0;
    char* const q = o.base + c * 16;
    u32x4 v[kRun / kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRun / kRows; ++j)
      v[j] = *reinterpret_cast<const u32x4*>(lds + (i * kRun + r0 + j * kRows) * kRow16<T> + c * 16);
#pragma unroll
    for (uint32_t j = 0; j < kRun / kRows; ++j)
      if (r0 + j * kRows < rows) *reinterpret_cast<u32x4*>(q + (r0 + j * kRows) * o.stride) = v[j];
  }
}

// ---------------------------------------------------------------------------
// Logits: M = vocabulary, N = tokens, K = dim.  A lane of an accumulator holds 4
// consecutive columns of one token.
//
// Forward: the tile's maximum m and sum s = sum exp(z - m) of every token, which
// k_loss merges as s = s1 exp(m1 - m) + s2 exp(m2 - m): 8 bytes a token and tile
// leave the chip instead of the logits.  One token, dim 768, 50257 rows: 17 us,
// 77 MB of weights at 4.5 TB/s; 2048 tokens, dim 4096: 738 us with its loss.
// Gradient: exp(z - lse) g in the storage type; the target's 1 is taken off
// where the tile holds it.
//
// In short steps the gradient's first workgroups copy the hidden rows for dweights,
// a row a wavefront, instead of a launch of their own (kRideTokens).
template <class E>
__device__ __forceinline__ void ride_rows(const LogitArgs& a, int* sm, int wave, int lane) {
  using S = typename E::S;
  int top = 0;
  if constexpr (__is_same(E, EF16)) {
    if (a.row_exp) {
      top = top_exponent<kWaves * 64>(a.row_exp, a.tokens, sm);
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.scale = top;
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < kRiderRows / kWaves; ++i) {
    const uint32_t t = blockIdx.x * kRiderRows + i * kWaves + wave;
    if (t >= a.grad_rows) break;
    const uint32_t col = t < a.tokens ? padded_col(a.sh, target_at(a.targets, a.target_bytes, t)) : kMasked;
    if (t < a.tokens && lane == 0) a.tcol[t] = col;
    const bool live = col != kMasked;
    float f = 1.f;
    if constexpr (__is_same(E, EF16)) f = live && a.row_exp ? row_factor(a.grad_loss[t], top) : 1.f;
    copy_row<E, 64>(reinterpret_cast<const S*>(static_cast<const char*>(a.x) + t * a.x_stride),
                    static_cast<char*>(a.xg) + t * a.x_stride, a.kbytes / sizeof(S), 16, lane, live, f);
  }
}

template <class E, class T, bool GRAD>
__global__ __launch_bounds__(kWaves * 64) void k_logits(LogitArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (GRAD && T::BN < 256) {
    if (blockIdx.x < a.riders) {
      ride_rows<E>(a, reinterpret_cast<int*>(lds), wave, lane);
      return;
    }
  }
  uint32_t tm, tn;
  tile_of(blockIdx.x - (GRAD && T::BN < 256 ? a.riders : 0), a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t cbase = a.c0 + tm * T::BM;
  const uint32_t t0 = tn * T::BN;

  KcShardLoader<T::BM> la;
  KcLoader<T::BN> lb;
  const uint32_t steps = (a.kbytes + 127) / 128;
  // Tiles of the vocabulary start at different places of their rows: rows are
  // often a power of two apart, and with every workgroup at the same place the
  // chip would read from a few memory channels at a time.  Eight tiles share a
  // start, as they share the tokens' rows in the L2.  (Loss of 128 x 4096 x 32000,
  // memory bound: 80 us with one start, 70 with these; 8192 x 4096 x 50257: the same.)
  const uint32_t kfirst = (tm / 8 * 2) % steps;
  la.init(a.sh, a.w_stride, cbase, a.c1, a.kbytes, kfirst, wave, lane);
  lb.init(a.x, a.x_stride, t0, a.tokens, a.kbytes, kfirst, steps, wave, lane);
  k_start<T>(lds, la, lb);
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, steps, acc, la, lb,
      [&](const char* t, int m, int s) { return frag_kc<E>(t, m0 + m * 32, s, lane); },
      [&](const char* t, int n, int s) { return frag_kc<E>(t, n0 + n * 32, s, lane); });

  // Column of register 4i + j of fragment m: lc + 32 m + 8 i + j.  Columns that pad
  // a slot have no logit; most tiles have none of them.
  const uint32_t cw = cbase + m0, half = (lane >> 5) * 4, lc = cw + half;
  uint32_t lim[T::MT];  // lc + 32 m + x exists for x < lim[m]
  bool full = true;
#pragma unroll
  for (int m = 0; m < T::MT; ++m) {
    const uint32_t c = cw + m * 32;
    uint32_t end = 0;
    for (int r = 0; r < a.sh.p; ++r)
      if (c >= a.sh.off[r] && c < a.sh.off[r + 1]) end = a.sh.off[r] + a.sh.rows[r];
    end = end < a.c1 ? end : a.c1;
    lim[m] = end > c + half ? end - (c + half) : 0;
    full = full && end >= c + 32;
  }
  if (!full) {
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int n = 0; n < T::NT; ++n)
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (static_cast<uint32_t>(x / 4 * 8 + x % 4) >= lim[m]) acc[m][n][x] = -__builtin_inff();
  }
  // The logit `rel` columns from lc in fragment column n, if this lane holds it.
  const auto pick = [&](int n, uint32_t rel, float& z) __attribute__((always_inline)) {
    bool here = false;
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (rel == static_cast<uint32_t>(m * 32 + x / 4 * 8 + x % 4)) {
          z = acc[m][n][x];
          here = true;
        }
    return here;
  };

  if constexpr (!GRAD) {
    float* red = reinterpret_cast<float*>(lds);  // [WM][BN][2]
#pragma unroll
    for (int n = 0; n < T::NT; ++n) {
      const uint32_t t = t0 + n0 + n * 32 + (lane & 31);
      float mx = -__builtin_inff();
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int x = 0; x < 16; ++x) mx = fmaxf(mx, acc[m][n][x]);
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      // a tile whose logits are all -inf has sum 0, not NaN
      const float ref = mx == -__builtin_inff() ? 0.f : mx;
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int x = 0; x < 16; ++x) sum += __expf(acc[m][n][x] - ref);
      sum += __shfl_xor(sum, 32);
      if (lane < 32) {
        float* q = red + (wm * T::BN + n0 + n * 32 + lane) * 2;
        q[0] = mx;
        q[1] = sum;
      }
      if (t < a.tokens) {
        const uint32_t col = padded_col(a.sh, target_at(a.targets, a.target_bytes, t));
        float z;
        if (col - cw < T::MT * 32 && pick(n, col - lc, z)) a.hit[t] = z;  // few tiles hold a token's target
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < T::BN; i += kWaves * 64) {
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
      const uint32_t tl = n0 + n * 32 + (lane & 31), t = t0 + tl;
      uint32_t col = kMasked;
      float lse = 0.f, g = 0.f;
      if (t < a.tokens) {
        col = T::BN < 256 && a.riders ? padded_col(a.sh, target_at(a.targets, a.target_bytes, t)) : a.tcol[t];
        lse = a.lse[t];
        g = a.grad_loss[t];
      }
      const uint32_t live = col != kMasked ? ~0u : 0u;
      if constexpr (__is_same(E, EF16)) g = ldexpf(g, 15 - token_exponent(g));
      float zt = 0.f;
      const bool hot = live && col - cw < T::MT * 32 && pick(n, col - lc, zt);
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = __expf(acc[m][n][4 * i + j] - lse) * g;
          if constexpr (sizeof(S) == 2) {
            put16<E, T>(lds, tl, m0 + m * 32 + i * 8 + half, v, live);
          } else {
            const uint32_t c = lc + m * 32 + i * 8;
            if (t < a.grad_rows && c < a.c1) {
              u32x4 w;
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[j]) & live;
              *reinterpret_cast<u32x4*>(static_cast<S*>(a.grad) + t * a.ld + (c - a.c0)) = w;
            }
          }
        }
      if (hot) {
        const float x = (__expf(zt - lse) - 1.f) * g;
        if constexpr (sizeof(S) == 2) {
          // The target's entry is the row's largest by far; what its rounding
          // takes goes into the two products on the side (HiddenRow,
          // k_weight_grad), which leaves the rounding of the outputs the
          // largest error.
          const uint32_t b = f32_to_half<E>(x);
          *reinterpret_cast<S*>(lds + tl * kRow16<T> + (col - cbase) * 2) = static_cast<S>(b);
          a.lo[t] = x - half_to_f32<E>(b);
        } else {
          static_cast<S*>(a.grad)[t * a.ld + (col - a.c0)] = x;
        }
      }
    }
    if constexpr (sizeof(S) == 2) {
      __syncthreads();
      take16<E, T>(lds, a.c1 - cbase, [&](uint32_t i) {
        const uint32_t t = t0 + i * 64;
        return OutRows{reinterpret_cast<char*>(static_cast<S*>(a.grad) + t * a.ld + (cbase - a.c0)), a.ld * sizeof(S),
                       t < a.grad_rows ? a.grad_rows - t : 0};
      });
    }
  }
}

// ---------------------------------------------------------------------------
// dhidden: M = dim, N = tokens, K = the piece's padded columns, in `splits`
// parts.  Where that is all of K the result is written, else float32 sums.
// Few tokens give few tiles and the whole vocabulary as K: split, it is read by
// the whole chip at once (96 x 768 x 50257 in float16: 42 parts, 27.6 us;
// their join rides on dweights' launch).
template <class E, class T>
__global__ __launch_bounds__(kWaves * 64) void k_hidden_grad(HiddenGradArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
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

  KsShardLoader<E, T::BM> la;
  KcLoader<T::BN> lb;
  la.init(a.sh, a.w_stride, static_cast<uint64_t>(d0) * esz, static_cast<uint64_t>(a.dim - d0) * esz,
          a.c0 + k_lo * Frag<E>::kBK, a.c0 + k_hi * Frag<E>::kBK, wave, lane);
  lb.init(a.grad, a.ld * esz, t0, a.grad_rows, (a.c1 - a.c0) * esz, k_lo, k_hi - k_lo, wave, lane);
  k_start<T>(lds, la, lb);
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, k_hi - k_lo, acc, la, lb,
      [&](const char* t, int m, int s) { return frag_ks<E, T::BM>(t, m0 + m * 32, s, lane); },
      [&](const char* t, int n, int s) { return frag_kc<E>(t, n0 + n * 32, s, lane); });
  using S = typename E::S;
  if (a.out) {
    // the whole vocabulary in one product: the result itself
#pragma unroll
    for (int n = 0; n < T::NT; ++n) {
      const uint32_t tl = n0 + n * 32 + (lane & 31), t = t0 + tl;
      const HiddenRow<E> h(a.sh, a.tcol, a.lo, a.grad_loss, t, a.tokens, a.dim);
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t dl = m0 + m * 32 + i * 8 + (lane >> 5) * 4, d = d0 + dl;
          float v[4] = {acc[m][n][4 * i], acc[m][n][4 * i + 1], acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
          if constexpr (esz == 2) {
            h.finish4(v, d, a.dim);
            put16<E, T>(lds, tl, dl, v, h.live ? ~0u : 0u);
          } else if (t < a.tokens && d < a.dim) {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = h.live ? __float_as_uint(v[j]) : 0u;
            *reinterpret_cast<u32x4*>(static_cast<S*>(a.out) + static_cast<uint64_t>(t) * a.dim + d) = w;
          }
        }
    }
    if constexpr (esz == 2) {
      __syncthreads();
      take16<E, T>(lds, a.dim - d0, [&](uint32_t i) {
        const uint32_t t = t0 + i * 64;
        return OutRows{reinterpret_cast<char*>(static_cast<S*>(a.out) + static_cast<uint64_t>(t) * a.dim + d0),
                       static_cast<uint64_t>(a.dim) * sizeof(S), t < a.tokens ? a.tokens - t : 0};
      });
    }
    return;
  }
  float* out = a.acc + split * a.split_stride;
  const bool vec = a.dim % 4 == 0;
#pragma unroll
  for (int n = 0; n < T::NT; ++n) {
    const uint32_t t = t0 + n0 + n * 32 + (lane & 31);
    if (t >= a.tokens) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = d0 + m0 + m * 32 + i * 8 + (lane >> 5) * 4;
        float* q = out + static_cast<uint64_t>(t) * a.dim + d;
        if (vec) {
          if (d < a.dim) {
            f32x4_t v = {acc[m][n][4 * i], acc[m][n][4 * i + 1], acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
            if (a.add) {
              const f32x4_t o = *reinterpret_cast<const f32x4_t*>(q);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] += o[j];
            }
            *reinterpret_cast<f32x4_t*>(q) = v;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d + j < a.dim) q[j] = a.add ? q[j] + acc[m][n][4 * i + j] : acc[m][n][4 * i + j];
        }
      }
  }
}

// The tokens of [b, b + kScan) whose target's padded column lies in [first, first +
// n) join `list`, which holds `have`, always in the same order.  The list takes
// 64 + kScan entries and 16 bytes more.
constexpr uint32_t kScan = 8 * kWaves * 64;

__device__ __forceinline__ void scan_targets(const uint32_t* tcol, uint32_t tokens, uint32_t b, uint32_t first,
                                             uint32_t n, uint32_t* list, uint32_t& have) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t* const found = list + 64 + kScan;
  uint64_t mask[8];
  uint32_t count = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t t = b + j * kWaves * 64 + threadIdx.x;
    const uint32_t c = t < tokens ? tcol[t] : kMasked;
    mask[j] = __ballot(c - first < n);  // kMasked - first is out of range
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) count += __popcll(mask[j]);
  if (lane == 0) found[wave] = count;
  __syncthreads();
  uint32_t at = have;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at += found[w];
    have += found[w];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (mask[j] >> lane & 1) list[at + __popcll(mask[j] & ((1ull << lane) - 1))] = b + j * kWaves * 64 + threadIdx.x;
    at += __popcll(mask[j]);
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// dweights: M = dim, N = the piece's padded columns, K = tokens.  With few tokens
// it is a write of the whole matrix (96 x 768 x 50257 in float16: 36 us for 77
// MB, most of it first loads and outputs of 2364 workgroups).
template <class E, class T>
__global__ __launch_bounds__(kWaves * 64) void k_weight_grad(WeightGradArgs a) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  using S = typename E::S;
  constexpr int esz = sizeof(S);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (T::BN < 256) {
    const uint32_t i = blockIdx.x - a.rider0;
    if (i < a.riders) {
      const uint32_t t = i / a.join_cols, by = i % a.join_cols;
      float* const part = reinterpret_cast<float*>(lds);
      if (t >= a.tokens) return;
      if (a.join.splits >= kJoinMany) join_block<E, 4, 4>(a.sh, a.join, t, by, part);
      else join_block<E, 1, 4>(a.sh, a.join, t, by, part);
      return;
    }
  }
  uint32_t tm, tn;
  tile_of(T::BN < 256 && a.rider0 == 0 ? blockIdx.x - a.riders : blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t d0 = tm * T::BM, v0 = tn * T::BN;
  KsLoader<E, T::BM> la;
  KsLoader<E, T::BN> lb;
  const char* const xg = static_cast<const char*>(a.xg) + static_cast<uint64_t>(d0) * esz;
  const uint64_t xg_cols = a.xg_stride - static_cast<uint64_t>(d0) * esz;
  la.init(xg, a.xg_stride, xg_cols, a.rows / Frag<E>::kBK, wave, lane);
  lb.init(static_cast<const char*>(a.grad) + static_cast<uint64_t>(v0) * esz, a.ld * esz,
          static_cast<uint64_t>(a.c1 - a.c0 - v0) * esz, a.rows / Frag<E>::kBK, wave, lane);
  k_start<T>(lds, la, lb);
  // What rounding took from the targets' entries (16-bit types): the tokens
  // whose target lies in this tile's columns are added as further K steps of up
  // to 64.  There are few, since the whole vocabulary shares the tokens: they are
  // looked up while the first loads arrive, and up to 64 of them wait in
  // registers for the end of the loop, one a lane with its column and remainder,
  // and this thread's chunks of their rows (2048 x 4096 x 32000: 549 us,
  // 545 without the remainders; 605 with all of it looked up at the end).  Tiles
  // with more of them, as text's commonest tokens give, look them up at the end
  // (gradient with targets as 1 / rank: 2048 x 4096 x 32000 1431 -> 1453 us, 8192 x
  // 4096 x 50257 8.16 -> 8.26 ms).
  const uint32_t first = a.c0 + v0;
  constexpr uint32_t RA = T::BM * esz, RB = T::BN * esz, kThreads = kWaves * 64;
  constexpr int NA = T::ABYTES / 16 / kThreads, NB = T::BBYTES / 16 / kThreads;
  uint32_t hits = 0, ecol = 0;
  float elo = 0.f;
  u32x4 rows[NA];
  const auto fetch = [&](const uint32_t* list, uint32_t n) __attribute__((always_inline)) {
    uint32_t t = 0;
    ecol = first;
    elo = 0.f;
    if (lane < static_cast<int>(n)) {
      t = list[lane];
      ecol = a.tcol[t];
      elo = a.lo[t];
    }
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      const uint32_t i = u * kThreads + threadIdx.x, k = i * 16 / RA;
      const uint32_t c = ks_chunk<E>(k, (i * 16 % RA) / 16) * 16;
      rows[u] = u32x4{0, 0, 0, 0};
      if (u * kThreads * 16 / RA < n) {
        const uint32_t tk = __shfl(t, static_cast<int>(k));
        if (k < n && c < xg_cols) rows[u] = *reinterpret_cast<const u32x4*>(xg + tk * a.xg_stride + c);
      }
    }
  };
  if constexpr (esz == 2) {
    uint32_t* const list = reinterpret_cast<uint32_t*>(lds + 2 * T::ABYTES);
    for (uint32_t b = 0; b < a.tokens && hits <= 64; b += kScan)
      scan_targets(a.tcol, a.tokens, b, first, T::BN, list, hits);
    hits = __builtin_amdgcn_readfirstlane(hits);
    fetch(list, hits <= 64 ? hits : 0);
  }
  f32x16_t acc[T::MT][T::NT];
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int m0 = wm * (T::MT * 32), n0 = wn * (T::NT * 32);
  k_loop<E, T>(
      lds, a.rows / Frag<E>::kBK, acc, la, lb,
      [&](const char* t, int m, int s) { return frag_ks<E, T::BM>(t, m0 + m * 32, s, lane); },
      [&](const char* t, int n, int s) { return frag_ks<E, T::BN>(t, n0 + n * 32, s, lane); });
  if constexpr (esz == 2) {
    // the tokens at hand, or, where there were too many, all of them again, 64 at a time
    uint32_t* const list = reinterpret_cast<uint32_t*>(lds + T::ABYTES);
    const bool held = hits <= 64;
    uint32_t have = 0, b = 0;
    for (;;) {
      uint32_t n = hits;
      if (!held) {
        while (have < 64 && b < a.tokens) {
          scan_targets(a.tcol, a.tokens, b, first, T::BN, list, have);
          b += kScan;
        }
        have = __builtin_amdgcn_readfirstlane(have);
        n = have < 64 ? have : 64;
        fetch(list, n);
      }
      if (n == 0) break;
      // A: the tokens' rows; B: in row k the remainder of token k in its column
      const uint32_t quarters = (n + 15) / 16;
      const uint32_t entry = (ecol - first) << 16 | f32_to_half<E>(elo);
#pragma unroll
      for (int u = 0; u < NA; ++u)
        if (u * kThreads * 16 / RA < quarters * 16)
          *reinterpret_cast<u32x4*>(lds + (u * kThreads + threadIdx.x) * 16) = rows[u];
#pragma unroll
      for (int u = 0; u < NB; ++u)
        if (u * kThreads * 16 / RB < quarters * 16) {
          const uint32_t i = u * kThreads + threadIdx.x, k = i * 16 / RB;
          const uint32_t e = __shfl(entry, static_cast<int>(k)), col = e >> 16;
          const uint32_t w = (e & 0xffffu) << (col % 2 * 16);
          const bool here = col / 8 == ks_chunk<E>(k, (i * 16 % RB) / 16);
          u32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = here && col % 8 / 2 == static_cast<uint32_t>(j) ? w : 0u;
          *reinterpret_cast<u32x4*>(lds + T::BOFF + i * 16) = v;
        }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (static_cast<uint32_t>(s) >= quarters) break;
        Frag<E> fa[T::MT], fb[T::NT];
#pragma unroll
        for (int m = 0; m < T::MT; ++m) fa[m] = frag_ks<E, T::BM>(lds, m0 + m * 32, s, lane);
#pragma unroll
        for (int n2 = 0; n2 < T::NT; ++n2) fb[n2] = frag_ks<E, T::BN>(lds + T::BOFF, n0 + n2 * 32, s, lane);
#pragma unroll
        for (int m = 0; m < T::MT; ++m)
#pragma unroll
          for (int n2 = 0; n2 < T::NT; ++n2) acc[m][n2] = mma<E>(fa[m], fb[n2], acc[m][n2]);
      }
      __syncthreads();
      if (held) break;
      have -= n;
      // the rest moves to the front, a workgroup's width at a time
      for (uint32_t i = 0; i < have; i += kThreads) {
        const uint32_t k = i + threadIdx.x;
        const uint32_t v = k < have ? list[64 + k] : 0;
        __syncthreads();
        if (k < have) list[k] = v;
        __syncthreads();
      }
    }
  }
  float scale = 1.f;
  if constexpr (__is_same(E, EF16)) scale = ldexpf(1.f, a.scale[0] - 30);
  // row n of the tile: a vocabulary row of one of the shards
  const auto row_of = [&](uint32_t n) -> S* {
    const uint32_t c = a.c0 + v0 + n;
    S* row = nullptr;
    if (c < a.c1)
      for (int r = 0; r < a.sh.p; ++r)
        if (c >= a.sh.off[r] && c - a.sh.off[r] < a.sh.rows[r])
          row = static_cast<S*>(a.dw[r]) + static_cast<uint64_t>(c - a.sh.off[r]) * a.dim;
    return row;
  };
  if (esz == 2 && a.vec) {
#pragma unroll
    for (int n = 0; n < T::NT; ++n)
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = acc[m][n][4 * i + j] * scale;
          if constexpr (esz == 2)
            put16<E, T>(lds, n0 + n * 32 + (lane & 31), m0 + m * 32 + i * 8 + (lane >> 5) * 4, v, ~0u);
        }
    __syncthreads();
    int r = 0;
    take16<E, T>(lds, a.dim - d0, [&](uint32_t i) {
      const uint32_t c = a.c0 + v0 + i * 64;  // a slot: rows of one shard
      if (c >= a.c1) return OutRows{nullptr, 0, 0};
      while (c >= a.sh.off[r + 1]) ++r;
      const uint32_t local = c - a.sh.off[r];
      return OutRows{reinterpret_cast<char*>(static_cast<S*>(a.dw[r]) + static_cast<uint64_t>(local) * a.dim + d0),
                     static_cast<uint64_t>(a.dim) * sizeof(S), a.sh.rows[r] > local ? a.sh.rows[r] - local : 0};
    });
    return;
  }
#pragma unroll
  for (int n = 0; n < T::NT; ++n) {
    S* row = row_of(n0 + n * 32 + (lane & 31));
    if (!row) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = d0 + m0 + m * 32 + i * 8 + (lane >> 5) * 4;
        if (esz == 4 && a.vec) {
          if (d < a.dim)
            *reinterpret_cast<f32x4_t*>(row + d) =
                f32x4_t{acc[m][n][4 * i], acc[m][n][4 * i + 1], acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d + j < a.dim) store_one<E>(row + d + j, acc[m][n][4 * i + j] * scale);
        }
      }
  }
}

// ---------------------------------------------------------------------------
// small_tile of the kind
template <class E>
using Small = std::conditional_t<sizeof(typename E::S) == 4, T64, T128>;

template <class E>
hipError_t run_logits(const LogitArgs& a, VocabTile t, bool grad, hipStream_t s) {
  const dim3 g(a.riders + a.tiles_m * a.tiles_n);
  if (g.x == 0) return hipSuccess;
#define RR_LAUNCH(TT)                                                        \
  if (grad)                                                                  \
    hipLaunchKernelGGL((k_logits<E, TT, true>), g, dim3(kWaves * 64), 0, s, a); \
  else                                                                       \
    hipLaunchKernelGGL((k_logits<E, TT, false>), g, dim3(kWaves * 64), 0, s, a);
  switch (t) {
    case VocabTile::k256x256: RR_LAUNCH(T256) break;
    case VocabTile::k128x32: RR_LAUNCH(T32) break;
    case VocabTile::k64x64: RR_LAUNCH(T64x64) break;
    default: RR_LAUNCH(Small<E>) break;
  }
#undef RR_LAUNCH
  return hipGetLastError();
}

template <class E>
hipError_t run_hidden_grad(const HiddenGradArgs& a, VocabTile t, hipStream_t s) {
  const dim3 g(a.tiles_m * a.tiles_n * a.splits);
  if (g.x == 0) return hipSuccess;
  switch (t) {
    case VocabTile::k256x256: hipLaunchKernelGGL((k_hidden_grad<E, T256>), g, dim3(kWaves * 64), 0, s, a); break;
    case VocabTile::k128x32: hipLaunchKernelGGL((k_hidden_grad<E, T32>), g, dim3(kWaves * 64), 0, s, a); break;
    default: hipLaunchKernelGGL((k_hidden_grad<E, Small<E>>), g, dim3(kWaves * 64), 0, s, a); break;
  }
  return hipGetLastError();
}

template <class E>
hipError_t run_weight_grad(const WeightGradArgs& a, VocabTile t, hipStream_t s) {
  const dim3 g(a.riders + a.tiles_m * a.tiles_n);
  if (g.x == 0) return hipSuccess;
  if (t == VocabTile::k256x256)
    hipLaunchKernelGGL((k_weight_grad<E, T256>), g, dim3(kWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((k_weight_grad<E, Small<E>>), g, dim3(kWaves * 64), 0, s, a);
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
