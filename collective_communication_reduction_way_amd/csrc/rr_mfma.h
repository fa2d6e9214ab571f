// rr_mfma.h -- tiles of matrix products on the matrix cores (gfx950): loads,
// LDS layouts, the K loop and the way out, shared by the vocabulary cross
// entropy's and the gated projections' kernels.
//
// acc[m][n] = sum_k A(m,k) B(n,k)
// with a BM x BN tile in the accumulators of 4 wavefronts.  An operand is
// staged in LDS in the layout it has in memory:
//   KC: rows are the M (or N) axis and k runs along a row (128 bytes a step);
//   KS: rows are the k axis and M (or N) runs along a row.  16-bit fragments of
//       such a tile are read with the transposing LDS load, so that no
//       operand is ever transposed in memory.
// Both layouts permute 16-byte chunks within a row by an XOR of row bits, so
// that the fragment reads hit all 64 banks (no conflicts counted); the
// permutation is applied to the global address, because the direct
// global-to-LDS load writes its 64 x 16 bytes consecutively.
#pragma once

#include "rr_device.h"

namespace rr {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

#define RR_LDS __attribute__((address_space(3)))

__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// A stretch of memory that a wavefront loads from, as a buffer descriptor: reads
// at or past `bytes` give zeros, which is how rows and columns that do not exist are
// read.  The same in every lane.
struct Span {
  u32x4 r;

  __device__ __forceinline__ void set(const char* base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(uniform(base));
    r = u32x4{static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32) & 0xFFFFu,
              static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(bytes)), 0x00027000u};
  }
  // The stretch begins `d` bytes further (negative: back).
  __device__ __forceinline__ void move(int64_t d) {
    const uint64_t p = (static_cast<uint64_t>(r[1]) << 32 | r[0]) + d;
    r[0] = static_cast<uint32_t>(p);
    r[1] = static_cast<uint32_t>(p >> 32);
  }
};
constexpr uint32_t kNoOffset = 0xFFFFFFF0u;  // past the end of every span

// A load may read a scalar register no sooner than five wait states after a vector
// instruction wrote it.  The compiler, which may form a descriptor's words in vector
// registers, sees to that for its own instructions, but not for load_to_lds.  So a
// changed span is fixed: whatever forms it stands in front of fix() and so of all
// inline assembly that follows, and between that and a load lie five instructions, or
// wait_for_spans() (k_start, k_loop).  16-bit times within 0.5 %, float32 steps up to 1 %
// more (with a wait at every change 0.6 and 2 %).
__device__ __forceinline__ void fix(Span& m) { asm volatile("" : "+s"(m.r)); }
template <int N>
__device__ __forceinline__ void fix(Span (&m)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) fix(m[i]);
}
__device__ __forceinline__ void wait_for_spans() { asm volatile("s_nop 4"); }

// LDS addresses are 32-bit numbers here: a generic pointer costs a second word and
// a comparison with null at every use.
__device__ __forceinline__ uint32_t lds_at(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((RR_LDS const char*)p));
}
template <class T>
__device__ __forceinline__ RR_LDS T* lds_ptr(uint32_t at) {
  return reinterpret_cast<RR_LDS T*>(static_cast<uintptr_t>(at));
}

// 16 bytes a lane from memory straight into LDS; `to` + `more` is the wavefront's base
// (more: a constant) and lane l's chunk lands 16 l further.  The instruction is written
// out because for the builtin the compiler waits for all loads in flight before
// the next transposing LDS read, whatever it reads.  Nothing comes back in
// registers; wait_for_loads() stands before the barrier after which the LDS is
// read.  (One wait state is due between the write of M0 and its use.)
__device__ __forceinline__ void load_to_lds(const Span& m, uint32_t offset, uint32_t to, int more) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is reserved: nothing of the compiler's lives in it
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset),
               "s"(m.r), "i"(more)
               : "m0", "scc");
#pragma clang diagnostic pop
}
__device__ __forceinline__ void wait_for_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// An LDS address of a lane, `tile` the same in all of them.  Written out so that it
// stays where it stands: left to itself the compiler forms all of a step's addresses
// in one run ahead of the products, and a run of more than eight instructions leaves
// the matrix cores idle (one wavefront a SIMD issues one instruction in four cycles,
// and a product takes 32; with runs of 20 to 40 at the step's start dhidden of 8192 x
// 4096 x 16384 took 1660 us, 1566 without).
__device__ __forceinline__ uint32_t lane_at(uint32_t tile, uint32_t offset) {
  uint32_t at;
  asm volatile("v_add_u32 %0, %1, %2" : "=v"(at) : "s"(tile), "v"(offset));
  return at;
}

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

// Fragment of rows r0 + 32 m .. r0 + 32 m + 31 of a KC tile, quarter s of the step.
template <class E>
__device__ __forceinline__ Frag<E> frag_kc(uint32_t tile, int r0, int m, int s, int lane) {
  const uint32_t row = r0 + (lane & 31);
  const uint32_t chunk = (s * 2 + (lane >> 5)) ^ ((lane >> 1) & 7);
  Frag<E> f;
  f.v = *lds_ptr<const u32x4>(lane_at(tile, row * 128 + chunk * 16) + m * 4096);
  return f;
}

// Fragment of columns c0 + 32 m .. c0 + 32 m + 31 of a KS tile of R columns.
template <class E, int R>
__device__ __forceinline__ Frag<E> frag_ks(uint32_t tile, int c0, int m, int s, int lane) {
  Frag<E> f;
  const uint32_t u = static_cast<uint32_t>(c0 >> 4) + 2 * m + ((lane >> 4) & 1);
  if constexpr (sizeof(typename E::S) == 2) {
    // 16 lanes read 4 rows of 16 columns and get a column of 4 rows each
    const uint32_t k = (lane >> 5) * 8 + ((lane >> 2) & 3);  // of the quarter
    const uint32_t q = lane_at(tile, k * (R * 2) + (u ^ ks_swizzle<E>(k)) * 32 + (lane & 3) * 8) + s * (16 * R * 2);
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4_t>(q));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4_t>(q + 4 * R * 2));
    const s16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    f.v = __builtin_bit_cast(u32x4, v);
  } else {
    const uint32_t k = (lane >> 5) * 4;
    const uint32_t q = lane_at(tile, k * (R * 4) + (u ^ ks_swizzle<E>(k)) * 64 + (lane & 15) * 4) + s * (8 * R * 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = *lds_ptr<const uint32_t>(q + j * (R * 4));
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
// to the row's start and up to `first` again, `steps` in all.  A span's bytes say
// which rows exist; they stay what they are while its base walks along the rows.
// The chunks of a row's last step that lie past its end are kept out by their
// lanes' offsets, which get the top bit for that step, past every span (a tile's
// rows span less than 2^31 bytes).
struct RowWalk {
  uint32_t pos, end, steps;  // bytes; the row's bytes in whole steps; steps left
  uint32_t flip;             // of this lane: 0 or the top bit
  bool any;                  // the last step is not whole

  __device__ __forceinline__ void init(uint32_t kbytes, uint32_t chunk, uint32_t first, uint32_t steps_) {
    end = __builtin_amdgcn_readfirstlane((kbytes + 127) / 128 * 128);
    pos = __builtin_amdgcn_readfirstlane(first * 128);
    steps = __builtin_amdgcn_readfirstlane(steps_);
    any = kbytes % 128 != 0;
    flip = end - 128 + chunk < kbytes ? 0u : 0x80000000u;
  }
  template <int N>
  __device__ __forceinline__ void turn(uint32_t (&off)[N]) const {
    if (pos + 128 == end) {
#pragma unroll
      for (int q = 0; q < N; ++q) off[q] ^= flip;
    }
  }
  template <int N, int M>
  __device__ __forceinline__ void start(uint32_t (&off)[N], Span (&m)[M]) const {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      m[i].move(pos);
      if (steps == 0) m[i].r[2] = 0;
    }
    fix(m);
    if (any) turn(off);
  }
  // On to the next step.  What few steps need stands behind branches that the compiler
  // may not turn into instructions of every step.
  template <int N, int M>
  __device__ __forceinline__ void advance(uint32_t (&off)[N], Span (&m)[M]) {
    const int32_t d = pos + 128 == end ? 128 - static_cast<int32_t>(end) : 128;
    if (any) {
      asm volatile("");
      turn(off);
      pos += d;
      turn(off);
      pos -= d;
    }
    pos += d;
    steps = __builtin_amdgcn_readfirstlane(steps ? steps - 1 : 0);
#pragma unroll
    for (int i = 0; i < M; ++i) m[i].move(d);
    if (steps == 0) {  // nothing is read after the last step
      asm volatile("");
#pragma unroll
      for (int i = 0; i < M; ++i) m[i].r[2] = 0;
    }
    fix(m);
  }
};

// KC over rows at a constant stride: rows row0 .. of a matrix of `rows` rows.
template <int R>
struct KcLoader {
  static constexpr int NQ = R / 8 / kWaves;
  uint32_t off[NQ];
  Span m[1];
  RowWalk w;
  uint32_t mine;  // the wavefront's place in a tile

  __device__ __forceinline__ void init(const void* src, uint64_t stride, uint32_t row0, uint32_t rows, uint32_t kbytes,
                                       uint32_t first, uint32_t steps, int wave, int lane) {
    mine = wave * 1024;
    const uint32_t chunk = kc_chunk(wave * 8 + (lane >> 3), lane & 7) * 16;
    const uint32_t n = row0 < rows ? (rows - row0 < R ? rows - row0 : R) : 0;
    m[0].set(static_cast<const char*>(src) + row0 * stride, n * static_cast<uint32_t>(stride));
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      off[q] = ((wave + q * kWaves) * 8 + (lane >> 3)) * static_cast<uint32_t>(stride) + chunk;
    w.init(kbytes, chunk, first, steps);
    w.start(off, m);
  }
  __device__ __forceinline__ void prepare() {}
  // Load q of the next step (zeros after the last one).
  __device__ __forceinline__ void load(int q, uint32_t lds) {
    load_to_lds(m[0], off[q], lds + mine, q * kWaves * 1024);
  }
  __device__ __forceinline__ void advance() { w.advance(off, m); }
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

// KS with rows at a constant stride, `rows` of them.
template <class E, int R>
struct KsLoader {
  static constexpr int NQ = KsOffsets<E, R>::NQ;
  KsOffsets<E, R> o;
  Span m;
  uint64_t stride;
  uint32_t tail;  // bytes of a row that belong to the tile's columns
  uint32_t rows;  // that are left
  uint32_t mine;

  __device__ __forceinline__ uint32_t bytes() const {
    const uint32_t n = rows < Frag<E>::kBK ? rows : Frag<E>::kBK;
    return __builtin_amdgcn_readfirstlane(n ? (n - 1) * static_cast<uint32_t>(stride) + tail : 0);
  }
  __device__ __forceinline__ void init(const char* src, uint64_t stride_, uint64_t cols, uint32_t rows_, int wave,
                                       int lane) {
    mine = wave * 1024;
    rows = __builtin_amdgcn_readfirstlane(rows_);
    stride = stride_;
    o.init(static_cast<uint32_t>(stride), cols, wave, lane);
    tail = static_cast<uint32_t>(cols < KsOffsets<E, R>::RB ? cols : KsOffsets<E, R>::RB);
    m.set(src, bytes());
    fix(m);
  }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void load(int q, uint32_t lds) {
    load_to_lds(m, o.off[q], lds + mine, q * kWaves * 1024);
  }
  __device__ __forceinline__ void advance() {
    rows = __builtin_amdgcn_readfirstlane(rows < Frag<E>::kBK ? 0 : rows - Frag<E>::kBK);
    m.move(Frag<E>::kBK * stride);
    m.r[2] = bytes();
    fix(m);
  }
};

// KS over shards' rows laid end to end, each padded to whole steps (SH: w, rows
// and off of a shard), padded rows [c, end): a step's rows are rows of one
// shard, rows past its end read zeros.
template <class E, int R, class SH>
struct KsShardLoader {
  static constexpr int NQ = KsOffsets<E, R>::NQ;
  KsOffsets<E, R> o;
  const SH* sh;
  uint64_t stride, col0;
  Span m;            // the next step's rows, at the tile's first column
  uint32_t rows;     // rows of the shard from there on
  uint32_t c, end;   // padded column of the next step; of the end
  uint32_t turn;     // where the next shard starts
  int r;
  uint32_t mine;

  __device__ __forceinline__ uint32_t bytes() const {
    const uint32_t n = rows < Frag<E>::kBK ? rows : Frag<E>::kBK;
    return __builtin_amdgcn_readfirstlane(
        n && c < end ? n * static_cast<uint32_t>(stride) - static_cast<uint32_t>(col0) : 0);
  }
  __device__ __forceinline__ void init(const SH& sh_, uint64_t stride_, uint64_t col0_, uint64_t cols, uint32_t c_,
                                       uint32_t end_, int wave, int lane) {
    mine = wave * 1024;
    sh = &sh_;
    stride = stride_;
    col0 = col0_;
    c = __builtin_amdgcn_readfirstlane(c_);
    end = __builtin_amdgcn_readfirstlane(end_);
    r = -1;
    turn = 0;
    rows = 0;
    m.set(nullptr, 0);
    fix(m);
    o.init(static_cast<uint32_t>(stride), cols, wave, lane);
  }
  // Before a step: the shard that holds it.
  __device__ __forceinline__ void prepare() {
    if (c >= turn && c < end) {
      do ++r;
      while (c >= sh->off[r + 1]);  // c < off[p]: ends at the shard that holds c
      const uint32_t local = c - sh->off[r];
      turn = __builtin_amdgcn_readfirstlane(sh->off[r + 1]);
      rows = __builtin_amdgcn_readfirstlane(sh->rows[r] > local ? sh->rows[r] - local : 0);
      m.set(static_cast<const char*>(sh->w[r]) + local * stride + col0, bytes());
      fix(m);
    }
  }
  __device__ __forceinline__ void load(int q, uint32_t lds) {
    load_to_lds(m, o.off[q], lds + mine, q * kWaves * 1024);
  }
  __device__ __forceinline__ void advance() {
    c += Frag<E>::kBK;
    rows = __builtin_amdgcn_readfirstlane(rows < Frag<E>::kBK ? 0 : rows - Frag<E>::kBK);
    m.move(Frag<E>::kBK * stride);
    m.r[2] = bytes();
    fix(m);
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
using T192 = Tile<256, 192, 2, 2>;
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
__device__ __forceinline__ void k_start(const char* mem, LA& la, LB& lb) {
  const uint32_t lds = lds_at(mem);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    la.prepare();
    wait_for_spans();
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
__device__ __forceinline__ void k_loop(const char* mem, uint32_t steps, f32x16_t (&acc)[T::MT][T::NT], LA& la, LB& lb,
                                       FA fa, FB fb) {
  const uint32_t lds = lds_at(mem);
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
  const auto read = [&](int to, int i, uint32_t ta, uint32_t tb, int s) __attribute__((always_inline)) {
    if (i < NT) b[to][i] = fb(tb, i, s);
    else if (i < NT + MT) a[to][i - NT] = fa(ta, i - NT, s);
  };
  const uint32_t lds_b = lds + T::BOFF;
  wait_for_all_but<LA::NQ + LB::NQ>();
  meet();
#pragma unroll
  for (int i = 0; i < NT + MT; ++i) read(0, i, lds, lds_b, 0);
  uint32_t slot = 0;  // of A: k mod 3
  for (uint32_t k = 0; k < steps; ++k) {
    const uint32_t slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot == 0 ? 2 : slot - 1;
    const uint32_t ac = lds + slot * T::ABYTES, an = lds + slot1 * T::ABYTES, af = lds + slot2 * T::ABYTES;
    const uint32_t bc = lds_b + (k & 1) * T::BBYTES, bn = lds_b + (~k & 1) * T::BBYTES;
    slot = slot1;
    la.prepare();
    // (otherwise a product and the addresses of MT + NT fragments or more stand before the first load)
    if constexpr (kMmas == 1) wait_for_spans();
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
        // loads past the last step read zeros, unused; where reads go between half of the
        // products the loads go between the others
        constexpr int kFree = kMmas - kFirst, kFrom = kFree ? kFirst : 0, kPer = kFree ? kFree : kMmas;
        if (i >= kFrom) {
          if (s < 3) {
            const int at = s * kPer + i - kFrom;
#pragma unroll
            for (int q = at * LA::NQ / (3 * kPer); q < (at + 1) * LA::NQ / (3 * kPer); ++q) la.load(q, af);
          } else {
#pragma unroll
            for (int q = (i - kFrom) * LB::NQ / kPer; q < (i - kFrom + 1) * LB::NQ / kPer; ++q) lb.load(q, bc);
          }
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

}  // namespace rr
