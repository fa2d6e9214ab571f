// rr_dropout.hip -- dropout from a counter-based generator on the way through
// the collectives (gfx950).
//
//   D(v)_i = word(i) >= threshold ? v * scale : +0,
//   word(i) = word i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw:
//   "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with key = seed and
//   counter = (floor(i/4), offset).
//
// The mask is a function of the element's index alone: no rank, launch shape
// or dtype changes it, and the gradient draws it again instead of reading it.
// One pass reads every input once and writes every output once; a block of
// the generator serves the 4 elements of a lane for all p ranks, and its 10
// rounds (two 32 x 32 -> 64 bit products each) run while the rank loads are in
// flight.  So every form is bound by memory: p = 8, 128 MiB of bfloat16 a rank, a
// residual a rank (3.22 GB) 568 us, 5.7 TB/s; the gather of 64 MiB 98 us, 6.2
// TB/s; a plain copy kernel of this library reaches 6.26 TB/s.
#include "rr_device.h"
#include "rr_kernels.h"

namespace rr {

namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// A kept value is scaled, a dropped one is zero whatever it was (infinities
// and NaN included).  The product and the residual addition are rounded one
// after the other, as separate operations.
__device__ __forceinline__ float drop_one(float v, uint32_t word, uint32_t threshold, float scale) {
#pragma clang fp contract(off)
  const float s = v * scale;
  return word >= threshold ? s : 0.f;
}
__device__ __forceinline__ float plus(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// k-th input of chunk c in ring order: c+1, c+2, ..., c (mod p).
__device__ __forceinline__ int ring_src(int k, int c, int p) {
  const int r = c + 1 + k;
  return r >= p ? r - p : r;
}

// 16-byte accesses at any element address: global memory takes them at any
// alignment, and a wavefront's 64 of them still cover whole lines but two.
template <class E, int V>
struct Group {
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2)));
  static_assert(V * sizeof(typename E::S) == 16, "one 16-byte access");
  __device__ __forceinline__ static void load(Raw<E, V>& r, const void* base, int64_t at) {
    r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const U*>(static_cast<const typename E::S*>(base) + at));
  }
  // (cached: the block is read again for the other destinations)
  __device__ __forceinline__ static void load_cached(Raw<E, V>& r, const void* base, int64_t at) {
    r.w[0] = *reinterpret_cast<const U*>(static_cast<const typename E::S*>(base) + at);
  }
  __device__ __forceinline__ static void store(void* base, int64_t at, const Raw<E, V>& r) {
    __builtin_nontemporal_store(static_cast<U>(r.w[0]), reinterpret_cast<U*>(static_cast<typename E::S*>(base) + at));
  }
};

// Which elements of a group stay, as bits.
template <int V>
__device__ __forceinline__ uint32_t keep_bits(const DropArgs& a, uint64_t offset, uint64_t group) {
  uint32_t keep = 0;
#pragma unroll
  for (int b = 0; b < V / 4; ++b) {
    const Words w = philox(group * (V / 4) + b, offset, a.seed);
#pragma unroll
    for (int j = 0; j < 4; ++j) keep |= (w.w[j] >= a.threshold ? 1u : 0u) << (b * 4 + j);
  }
  return keep;
}

template <int V>
__device__ __forceinline__ void drop_bits(float* v, uint32_t keep, float scale) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = drop_one(v[j], keep >> j & 1, 1u, scale);
}

template <int V>
__device__ __forceinline__ void add_to(float* a, const float* b) {
#pragma unroll
  for (int j = 0; j < V; ++j) a[j] = plus(a[j], b[j]);
}

// Groups a lane handles at once, and ranks whose loads it keeps in flight.  The
// folds: two groups of eight ranks and their residuals; measured at p = 8, 128
// MiB a rank in bfloat16 with a residual a rank, one group of four ranks at a
// time 615 us, two of eight 557 us, four of eight 551 us (and one workgroup
// less a compute unit for shorter vectors); the rounds with grid barriers that
// serve the plain all-reduce lost here (585 us and more: a lane has to hold p
// results instead of one, so a round is short).
template <DropForm F>
constexpr int kGroups = F == DropForm::kRanks ? 4 : F == DropForm::kGather ? 1 : 2;
constexpr int kRanksAtOnce = 8;

// U whole groups of chunk `seg`, the lane's first one `g`, kBlock apart; P: the
// ranks, 0 = a.p; in0 / out0: the element of the full vector at which the inputs / outputs start.
template <class E, DropForm F, int U, int P>
__device__ __forceinline__ void drop_groups(const DropArgs& a, uint64_t offset, int seg, uint64_t g, uint64_t in0,
                                            uint64_t out0) {
  constexpr int V = 16 / static_cast<int>(sizeof(typename E::S));
  using G = Group<E, V>;
  const int p = P > 0 ? P : a.p;
  const int64_t ii = static_cast<int64_t>(g * V - in0), io = static_cast<int64_t>(g * V - out0);
  constexpr int64_t kStep = kBlock * V;
  uint32_t keep[U];
  if constexpr (F == DropForm::kRanks) {
    constexpr int B = 4;
    bool first = true;
    for (int r0 = 0; r0 < p; r0 += B) {
      Raw<E, V> x[B][U], z[B][U];
#pragma unroll
      for (int k = 0; k < B; ++k)
        if (r0 + k < p)
#pragma unroll
          for (int u = 0; u < U; ++u) G::load(x[k][u], a.in[r0 + k], ii + u * kStep);
      if (a.has_res)
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (r0 + k < p)
#pragma unroll
            for (int u = 0; u < U; ++u) G::load(z[k][u], a.res[r0 + k], io + u * kStep);
      if (first)
#pragma unroll
        for (int u = 0; u < U; ++u) keep[u] = keep_bits<V>(a, offset, g + u * kBlock);
      first = false;
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (r0 + k >= p) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[V];
          unpack(x[k][u], v);
          drop_bits<V>(v, keep[u], a.scale);
          if (a.has_res) {
            float w[V];
            unpack(z[k][u], w);
            add_to<V>(v, w);
          }
          pack(v, x[k][u]);
          G::store(a.out[r0 + k], io + u * kStep, x[k][u]);
        }
      }
    }
  } else if constexpr (F == DropForm::kGather) {
    Raw<E, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) G::load_cached(x[u], a.in[seg], ii + u * kStep);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[V];
      keep[u] = keep_bits<V>(a, offset, g + u * kBlock);
      unpack(x[u], v);
      drop_bits<V>(v, keep[u], a.scale);
      pack(v, x[u]);
    }
    for (int r = 0; r < p; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) G::store(a.out[r], io + u * kStep, x[u]);
  } else {
    constexpr int B = kRanksAtOnce;
    constexpr bool kAll = F == DropForm::kReduce;
    Raw<E, V> x[B][U], z[B][U];
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (k < p)
#pragma unroll
        for (int u = 0; u < U; ++u) G::load(x[k][u], a.in[ring_src(k, seg, p)], ii + u * kStep);
    // the residuals of the first outputs: one where all share it
    const int nres = !a.has_res ? 0 : !kAll || a.one_res ? 1 : p;
#pragma unroll
    for (int k = 0; k < (kAll ? B : 1); ++k)
      if (k < nres)
#pragma unroll
        for (int u = 0; u < U; ++u) G::load(z[k][u], a.res[kAll ? k : seg], io + u * kStep);
#pragma unroll
    for (int u = 0; u < U; ++u) keep[u] = keep_bits<V>(a, offset, g + u * kBlock);
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) unpack(x[0][u], acc[u]);
#pragma unroll
    for (int k = 1; k < B; ++k) {
      if (k >= p) break;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[V];
        unpack(x[k][u], v);
        add_to<V>(acc[u], v);
      }
    }
    for (int k0 = B; k0 < p; k0 += B) {
#pragma unroll
      for (int k = 0; k < B; ++k)
        if (k0 + k < p)
#pragma unroll
          for (int u = 0; u < U; ++u) G::load(x[k][u], a.in[ring_src(k0 + k, seg, p)], ii + u * kStep);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (k0 + k >= p) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[V];
          unpack(x[k][u], v);
          add_to<V>(acc[u], v);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) drop_bits<V>(acc[u], keep[u], a.scale);
    if (nres <= 1) {
      // one result for every output
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (nres == 1) {
          float w[V];
          unpack(z[0][u], w);
          add_to<V>(acc[u], w);
        }
        pack(acc[u], x[0][u]);
      }
      if constexpr (kAll) {
        for (int r = 0; r < p; ++r)
#pragma unroll
          for (int u = 0; u < U; ++u) G::store(a.out[r], io + u * kStep, x[0][u]);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) G::store(a.out[seg], io + u * kStep, x[0][u]);
      }
    } else {
      for (int r0 = 0; r0 < p; r0 += B) {
        if (r0 > 0)
#pragma unroll
          for (int k = 0; k < B; ++k)
            if (r0 + k < p)
#pragma unroll
              for (int u = 0; u < U; ++u) G::load(z[k][u], a.res[r0 + k], io + u * kStep);
#pragma unroll
        for (int k = 0; k < B; ++k) {
          if (r0 + k >= p) break;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float w[V];
            unpack(z[k][u], w);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = plus(acc[u][j], w[j]);
            pack(w, z[k][u]);
            G::store(a.out[r0 + k], io + u * kStep, z[k][u]);
          }
        }
      }
    }
  }
}

// Elements [e0, e1) of chunk `seg`, fewer than a group: one by one, the mask's
// block drawn for each.
template <class E, DropForm F>
__device__ void drop_ends(const DropArgs& a, uint64_t offset, int seg, uint64_t e0, uint64_t e1, uint64_t in0,
                          uint64_t out0) {
  using S = typename E::S;
  const int p = a.p;
  const auto in = [&](int r, uint64_t e) { return load_one<E>(static_cast<const S*>(a.in[r]) + (e - in0)); };
  const auto res = [&](int r, uint64_t e) { return load_one<E>(static_cast<const S*>(a.res[r]) + (e - out0)); };
  const auto out = [&](int r, uint64_t e, float v) { store_one<E>(static_cast<S*>(a.out[r]) + (e - out0), v); };
  for (uint64_t e = e0; e < e1; ++e) {
    const Words w = philox(e / 4, offset, a.seed);
    const uint32_t sel = static_cast<uint32_t>(e & 3);
    const uint32_t word = sel == 0 ? w.w[0] : sel == 1 ? w.w[1] : sel == 2 ? w.w[2] : w.w[3];
    const auto drop = [&](float v) { return drop_one(v, word, a.threshold, a.scale); };
    if constexpr (F == DropForm::kRanks) {
      for (int r = 0; r < p; ++r) {
        const float v = drop(in(r, e));
        out(r, e, a.has_res ? plus(v, res(r, e)) : v);
      }
    } else if constexpr (F == DropForm::kGather) {
      const float v = drop(in(seg, e));
      for (int r = 0; r < p; ++r) out(r, e, v);
    } else {
      float v = in(ring_src(0, seg, p), e);
      for (int k = 1; k < p; ++k) v = plus(v, in(ring_src(k, seg, p), e));
      v = drop(v);
      if constexpr (F == DropForm::kScatter) {
        out(seg, e, a.has_res ? plus(v, res(seg, e)) : v);
      } else if (a.one_res) {
        if (a.has_res) v = plus(v, res(0, e));
        for (int r = 0; r < p; ++r) out(r, e, v);
      } else {
        for (int r = 0; r < p; ++r) out(r, e, a.has_res ? plus(v, res(r, e)) : v);
      }
    }
  }
}

// The groups of a chunk: those that touch it.  Groups start at multiples of V
// of the full vector, so that a group holds whole blocks of the generator; the
// first and the last one may hold elements of other chunks.
struct ChunkGroups {
  uint64_t lo, hi, g0, groups;
};
template <int V>
__device__ __forceinline__ ChunkGroups chunk_groups(const DropArgs& a, int seg) {
  const uint64_t lo = a.bound[seg], hi = a.bound[seg + 1];
  return ChunkGroups{lo, hi, lo / V, hi > lo ? (hi + V - 1) / V - lo / V : 0};
}

// Workgroup row y = chunk; along x the workgroups stride over the chunk's
// tiles of kBlock*U groups.
template <class E, DropForm F, int U, int P>
__global__ __launch_bounds__(kBlock) void k_dropout(DropArgs a) {
  constexpr int V = 16 / static_cast<int>(sizeof(typename E::S));
  constexpr uint64_t kTile = static_cast<uint64_t>(kBlock) * U;
  const int seg = blockIdx.y;
  const ChunkGroups c = chunk_groups<V>(a, seg);
  // a sharded side is addressed from the chunk's start
  const uint64_t in0 = F == DropForm::kGather ? c.lo : 0, out0 = F == DropForm::kScatter ? c.lo : 0;
  const uint64_t offset = a.offset + (a.offset_dev ? *a.offset_dev : 0);
  for (uint64_t t = blockIdx.x; t * kTile < c.groups; t += gridDim.x) {
    const uint64_t first = c.g0 + t * kTile;  // the tile's first group
    if (first * V >= c.lo && (first + kTile) * V <= c.hi) {
      drop_groups<E, F, U, P>(a, offset, seg, first + threadIdx.x, in0, out0);
      continue;
    }
    for (int u = 0; u < U; ++u) {
      const uint64_t g = first + u * kBlock + threadIdx.x;
      const uint64_t e0 = g * V > c.lo ? g * V : c.lo, e1 = (g + 1) * V < c.hi ? (g + 1) * V : c.hi;
      if (e0 >= e1) continue;
      if (e1 - e0 == V) drop_groups<E, F, 1, P>(a, offset, seg, g, in0, out0);
      else drop_ends<E, F>(a, offset, seg, e0, e1, in0, out0);
    }
  }
}

// The all-gather form laid out for the XCDs, as the plain all-gather above 128
// MiB written (rr_copy.hip, k_fanout_xcd): a workgroup drops one block of kBlock
// groups and writes it to D destinations; the workgroups of an XCD take W blocks
// for one group of destinations, then the same blocks for the next, so that a
// block comes from HBM once.  The mask is drawn once for each group of
// destinations.  Measured, p = 8, 64 MiB of bfloat16 gathered: 136 us with every
// destination written by one workgroup, 92 us with D = 2, 102 with 4, 162 with 1
// (W = 64; 4 and 16 within 3%).
constexpr int kXcds = 8;
constexpr int kGatherD = 2;
constexpr uint32_t kGatherW = 64;
constexpr uint64_t kGatherXcdBytes = 128ull << 20;

template <class E>
__global__ __launch_bounds__(kBlock) void k_gather_xcd(DropArgs a, uint32_t blocks_per_chunk, uint32_t blocks) {
  constexpr int V = 16 / static_cast<int>(sizeof(typename E::S));
  const uint32_t x = blockIdx.x % kXcds, j = blockIdx.x / kXcds;
  const uint32_t G = (static_cast<uint32_t>(a.p) + kGatherD - 1) / kGatherD;
  const uint32_t v = j / (G * kGatherW), rem = j - v * G * kGatherW, d = rem / kGatherW;
  const uint32_t b = (v * kGatherW + (rem - d * kGatherW)) * kXcds + x;
  if (b >= blocks) return;
  const int seg = static_cast<int>(b / blocks_per_chunk);
  const ChunkGroups c = chunk_groups<V>(a, seg);
  const uint64_t i = static_cast<uint64_t>(b - seg * blocks_per_chunk) * kBlock + threadIdx.x;
  if (i >= c.groups) return;
  const uint64_t g = c.g0 + i;
  const uint64_t offset = a.offset + (a.offset_dev ? *a.offset_dev : 0);
  const int r0 = static_cast<int>(d) * kGatherD, r1 = r0 + kGatherD < a.p ? r0 + kGatherD : a.p;
  const uint64_t e0 = g * V > c.lo ? g * V : c.lo, e1 = (g + 1) * V < c.hi ? (g + 1) * V : c.hi;
  using S = typename E::S;
  if (e1 - e0 == V) {
    Raw<E, V> q;
    Group<E, V>::load_cached(q, a.in[seg], static_cast<int64_t>(g * V - c.lo));
    const uint32_t keep = keep_bits<V>(a, offset, g);
    float f[V];
    unpack(q, f);
    drop_bits<V>(f, keep, a.scale);
    pack(f, q);
    for (int r = r0; r < r1; ++r) Group<E, V>::store(a.out[r], static_cast<int64_t>(g * V), q);
  } else {
    for (uint64_t e = e0; e < e1; ++e) {
      const uint32_t keep = keep_bits<V>(a, offset, g) >> (e - g * V) & 1;
      const float f = drop_one(load_one<E>(static_cast<const S*>(a.in[seg]) + (e - c.lo)), keep, 1u, a.scale);
      for (int r = r0; r < r1; ++r) store_one<E>(static_cast<S*>(a.out[r]) + e, f);
    }
  }
}

template <class E, DropForm F>
hipError_t run_form(const DropArgs& a, uint64_t longest, hipStream_t s) {
  constexpr int U = kGroups<F>;
  // Vectors that leave compute units idle take one group a lane.
  const bool few = longest * a.chunks < static_cast<uint64_t>(U) * kBlock * 256;
  const uint64_t tile = static_cast<uint64_t>(kBlock) * (few ? 1 : U);
  const uint64_t wg = (longest + tile - 1) / tile;
  constexpr uint64_t kMaxX = 1u << 20;  // longer chunks stride
  const dim3 grid(static_cast<uint32_t>(wg < kMaxX ? wg : kMaxX), static_cast<uint32_t>(a.chunks));
  if (few) {
    hipLaunchKernelGGL((k_dropout<E, F, 1, 0>), grid, dim3(kBlock), 0, s, a);
    return hipGetLastError();
  }
  // The folds of eight and four ranks are compiled for them: with the rank count
  // known, all loads of a lane go out in one block (p = 8, as above: 591 us with
  // the count at run time).
  if constexpr (F == DropForm::kReduce || F == DropForm::kScatter) {
    if (a.p == 8 || a.p == 4) {
      if (a.p == 8)
        hipLaunchKernelGGL((k_dropout<E, F, U, 8>), grid, dim3(kBlock), 0, s, a);
      else
        hipLaunchKernelGGL((k_dropout<E, F, U, 4>), grid, dim3(kBlock), 0, s, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_dropout<E, F, U, 0>), grid, dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <class E>
hipError_t run_dropout(const DropArgs& a, DropForm f, hipStream_t s) {
  constexpr uint64_t V = 16 / sizeof(typename E::S);
  uint64_t longest = 0;
  for (int c = 0; c < a.chunks; ++c) {
    const uint64_t groups = (a.bound[c + 1] + V - 1) / V - a.bound[c] / V;
    if (a.bound[c + 1] > a.bound[c] && groups > longest) longest = groups;
  }
  if (longest == 0) return hipSuccess;
  switch (f) {
    case DropForm::kReduce: return run_form<E, DropForm::kReduce>(a, longest, s);
    case DropForm::kScatter: return run_form<E, DropForm::kScatter>(a, longest, s);
    case DropForm::kRanks: return run_form<E, DropForm::kRanks>(a, longest, s);
    default: break;
  }
  const uint64_t per = (longest + kBlock - 1) / kBlock, blocks = per * a.chunks;
  const uint64_t dst = (static_cast<uint64_t>(a.p) + kGatherD - 1) / kGatherD;
  const uint64_t windows = ((blocks + kXcds - 1) / kXcds + kGatherW - 1) / kGatherW;
  const uint64_t grid = windows * kGatherW * dst * kXcds;
  const uint64_t written = a.bound[a.chunks] * sizeof(typename E::S) * static_cast<uint64_t>(a.p);
  // In place a workgroup would drop the shard under the others that still read
  // it: there one workgroup writes every destination.
  bool in_place = false;
  for (int c = 0; c < a.chunks; ++c)
    in_place = in_place || a.in[c] == static_cast<const char*>(a.out[c]) + a.bound[c] * sizeof(typename E::S);
  if (written > kGatherXcdBytes && !in_place && grid * kBlock < (1ull << 32)) {
    hipLaunchKernelGGL(k_gather_xcd<E>, dim3(static_cast<uint32_t>(grid)), dim3(kBlock), 0, s, a,
                       static_cast<uint32_t>(per), static_cast<uint32_t>(blocks));
    return hipGetLastError();
  }
  return run_form<E, DropForm::kGather>(a, longest, s);
}

}  // namespace

hipError_t launch_dropout(const DropArgs& a, DropForm f, Kind k, hipStream_t s) {
  switch (k) {
    case Kind::kF32: return run_dropout<EF32>(a, f, s);
    case Kind::kBF16: return run_dropout<EBF16>(a, f, s);
    default: return run_dropout<EF16>(a, f, s);
  }
}

}  // namespace rr
