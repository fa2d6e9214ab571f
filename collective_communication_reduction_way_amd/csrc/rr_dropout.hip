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
// flight.
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

// Ranks whose loads a lane keeps in flight.
constexpr int kBatch = 4;

// One group of V elements of chunk `seg`, first element i of the full vector,
// at element `ii` of the inputs and `io` of the outputs.  VEC: whole groups in
// 16-byte accesses; else elements j0 .. j1-1 of the group, one by one (ii and
// io may then lie before their buffer's start).
template <class E, DropForm F, int V, bool VEC>
__device__ __forceinline__ void drop_group(const DropArgs& a, uint64_t offset, int seg, uint64_t i, int64_t ii,
                                           int64_t io, int j0, int j1) {
  using S = typename E::S;
  const int p = a.p;
  auto load = [&](float* v, const void* base, int64_t at) {
    const S* b = static_cast<const S*>(base);
    if constexpr (VEC) {
      Raw<E, V> r;
      load_group<true>(r, b + at);
      unpack(r, v);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = j >= j0 && j < j1 ? load_one<E>(b + (at + j)) : 0.f;
    }
  };
  auto store = [&](void* base, int64_t at, const float* v) {
    S* b = static_cast<S*>(base);
    if constexpr (VEC) {
      Raw<E, V> r;
      pack(v, r);
      store_group<true>(b + at, r);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j >= j0 && j < j1) store_one<E>(b + (at + j), v[j]);
    }
  };
  // the mask of the group: V/4 blocks of the generator
  auto mask = [&](float* v) {
#pragma unroll
    for (int b = 0; b < V / 4; ++b) {
      const Words w = philox(i / 4 + b, offset, a.seed);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[b * 4 + j] = drop_one(v[b * 4 + j], w.w[j], a.threshold, a.scale);
    }
  };

  if constexpr (F == DropForm::kRanks) {
    uint32_t keep = 0;  // the mask once for all ranks
#pragma unroll
    for (int b = 0; b < V / 4; ++b) {
      const Words w = philox(i / 4 + b, offset, a.seed);
#pragma unroll
      for (int j = 0; j < 4; ++j) keep |= (w.w[j] >= a.threshold ? 1u : 0u) << (b * 4 + j);
    }
    for (int r0 = 0; r0 < p; r0 += kBatch) {
      float v[kBatch][V], res[kBatch][V];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (r0 + k < p) load(v[k], a.in[r0 + k], ii);
      if (a.has_res) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (r0 + k < p) load(res[k], a.res[r0 + k], ii);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (r0 + k >= p) break;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[k][j] = drop_one(v[k][j], keep >> j & 1, 1u, a.scale);
          if (a.has_res) v[k][j] = plus(v[k][j], res[k][j]);
        }
        store(a.out[r0 + k], io, v[k]);
      }
    }
  } else if constexpr (F == DropForm::kGather) {
    float v[V];
    load(v, a.in[seg], ii);
    mask(v);
    for (int r = 0; r < p; ++r) store(a.out[r], io, v);
  } else {
    float acc[V];
    load(acc, a.in[ring_src(0, seg, p)], ii);
    for (int k0 = 1; k0 < p; k0 += kBatch) {
      float v[kBatch][V];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < p) load(v[k], a.in[ring_src(k0 + k, seg, p)], ii);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k >= p) break;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = plus(acc[j], v[k][j]);
      }
    }
    mask(acc);
    if constexpr (F == DropForm::kScatter) {
      if (a.has_res) {
        float res[V];
        load(res, a.res[seg], io);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = plus(acc[j], res[j]);
      }
      store(a.out[seg], io, acc);
    } else {
      if (!a.has_res) {
        for (int r = 0; r < p; ++r) store(a.out[r], io, acc);
      } else if (a.one_res) {
        float res[V];
        load(res, a.res[0], io);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = plus(acc[j], res[j]);
        for (int r = 0; r < p; ++r) store(a.out[r], io, acc);
      } else {
        for (int r0 = 0; r0 < p; r0 += kBatch) {
          float res[kBatch][V];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (r0 + k < p) load(res[k], a.res[r0 + k], io);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (r0 + k >= p) break;
#pragma unroll
            for (int j = 0; j < V; ++j) res[k][j] = plus(acc[j], res[k][j]);
            store(a.out[r0 + k], io, res[k]);
          }
        }
      }
    }
  }
}

// Workgroup row y = chunk; along x the workgroups stride over the chunk's
// groups.  Groups start at multiples of V of the full vector, so that a group
// holds whole blocks of the generator; a chunk's ragged ends are groups with
// fewer elements, moved one by one.
template <class E, DropForm F>
__global__ __launch_bounds__(kBlock) void k_dropout(DropArgs a) {
  constexpr int V = 16 / static_cast<int>(sizeof(typename E::S));
  const int seg = blockIdx.y;
  const uint64_t lo = a.bound[seg], hi = a.bound[seg + 1];
  // a sharded side is addressed from the chunk's start
  const uint64_t in0 = F == DropForm::kGather ? lo : 0, out0 = F == DropForm::kScatter ? lo : 0;
  const uint64_t offset = a.offset + (a.offset_dev ? *a.offset_dev : 0);
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * kBlock;
  for (uint64_t g = lo / V + static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; g * V < hi; g += stride) {
    const uint64_t i = g * V;
    const int64_t ii = static_cast<int64_t>(i - in0), io = static_cast<int64_t>(i - out0);
    if (a.vec && i >= lo && i + V <= hi) {
      drop_group<E, F, V, true>(a, offset, seg, i, ii, io, 0, V);
    } else {
      const int j0 = i < lo ? static_cast<int>(lo - i) : 0;
      const int j1 = i + V > hi ? static_cast<int>(hi - i) : V;
      drop_group<E, F, V, false>(a, offset, seg, i, ii, io, j0, j1);
    }
  }
}

template <class E>
hipError_t run_dropout(const DropArgs& a, DropForm f, dim3 grid, hipStream_t s) {
  switch (f) {
    case DropForm::kReduce: hipLaunchKernelGGL((k_dropout<E, DropForm::kReduce>), grid, dim3(kBlock), 0, s, a); break;
    case DropForm::kScatter: hipLaunchKernelGGL((k_dropout<E, DropForm::kScatter>), grid, dim3(kBlock), 0, s, a); break;
    case DropForm::kGather: hipLaunchKernelGGL((k_dropout<E, DropForm::kGather>), grid, dim3(kBlock), 0, s, a); break;
    default: hipLaunchKernelGGL((k_dropout<E, DropForm::kRanks>), grid, dim3(kBlock), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropArgs& a, DropForm f, Kind k, hipStream_t s) {
  const uint64_t V = k == Kind::kF32 ? 4 : 8;
  uint64_t longest = 0;
  for (int c = 0; c < a.chunks; ++c) {
    const uint64_t groups = (a.bound[c + 1] + V - 1) / V - a.bound[c] / V;
    if (a.bound[c + 1] > a.bound[c] && groups > longest) longest = groups;
  }
  if (longest == 0) return hipSuccess;
  const uint64_t wg = (longest + kBlock - 1) / kBlock;
  constexpr uint64_t kMaxX = 1u << 17;  // longer chunks stride
  const dim3 grid(static_cast<uint32_t>(wg < kMaxX ? wg : kMaxX), static_cast<uint32_t>(a.chunks));
  switch (k) {
    case Kind::kF32: return run_dropout<EF32>(a, f, grid, s);
    case Kind::kBF16: return run_dropout<EBF16>(a, f, grid, s);
    default: return run_dropout<EF16>(a, f, grid, s);
  }
}

}  // namespace rr
