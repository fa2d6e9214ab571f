// rr_gated.h -- plan and argument blocks of the gated column-parallel
// projections (internal to librr.so).
//
// The F features are cut over the p virtual ranks at the chunk bounds
// floor(r*F/p).  The kernels work in "padded features": every shard's features
// rounded up to a multiple of kFeat, the shards laid end to end.  The gradients
// of both projections lie in one matrix of twice as many columns: kFeat columns
// of the gate, the same kFeat of the up projection, and so on, so that a run of
// kFeat columns reads one shard of one weight.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "rr.h"
#include "rr_kernels.h"

namespace rr {

constexpr uint32_t kFeat = 64;

struct GatedShards {
  const void* gate[RR_MAX_RANKS];   // row 0 of each shard's [rows, dim] matrices
  const void* up[RR_MAX_RANKS];
  uint32_t off[RR_MAX_RANKS + 1];   // first padded feature of each shard; off[p] = all of them
  uint32_t rows[RR_MAX_RANKS];      // the shard's own features
  int32_t p;
};

enum class GatedAct : int { kSilu = 0, kGelu = 1 };

// Tile of the matrix products: (M axis) x (N axis).  k128x64: float32 only; k128x32:
// dhidden only; k64x64: forward only; k256x192: forward, 16-bit types only; kFew: k_gated_few, 16 features and up to 128
// tokens a workgroup, forward only.
enum class GatedTile : int { k256x256 = 0, k128x128 = 1, k128x64 = 2, k128x32 = 3, k64x64 = 4, kFew = 5, k256x192 = 6 };
constexpr uint32_t tile_m(GatedTile t) {
  return t == GatedTile::k256x256 || t == GatedTile::k256x192 ? 256 : t == GatedTile::k64x64 ? 64 : 128;
}
constexpr uint32_t tile_n(GatedTile t) {
  switch (t) {
    case GatedTile::k256x256: return 256;
    case GatedTile::k256x192: return 192;
    case GatedTile::k128x64: return 64;
    case GatedTile::k64x64: return 64;
    case GatedTile::k128x32: return 32;
    default: return 128;
  }
}

// What the forward kernels write for the padded features [f0, f1):
//   kForward: h = act(A) U, and the products A = x gate^T, U = x up^T themselves where
//     they are kept: in a and u, or in the matrix `pre` of kFeat-column runs;
//   kGrad: the products' gradients, from dh, into `pre` in the storage type (columns
//     that pad a run are zeros).
enum class GatedMode : int { kForward = 0, kGrad = 1 };
struct GatedArgs {
  GatedShards sh;
  void* h[RR_MAX_RANKS];   // [tokens, rows[r]]; kGrad: dh, read
  void* a[RR_MAX_RANKS];   // [tokens, rows[r]] each
  void* u[RR_MAX_RANKS];
  void* pre;               // NULL, or [tokens][pre_ld]
  uint64_t pre_ld;
  const void* x;           // [tokens, dim] rows of x_stride bytes
  uint64_t x_stride;
  uint64_t w_stride;
  uint32_t kbytes;         // dim * element size; but for kFew a multiple of 16
  uint32_t dim;
  uint32_t tokens;
  uint32_t f0, f1;
  uint32_t tiles_m, tiles_n;
  int32_t has_h, has_pre;
  int32_t pre32;           // kept products are float32 (else of the storage type)
};

// The gradients of the two products, into `grad` (columns that pad a run are
// zeros), from dh and the products: a and u, or `pre`.
struct GatedGradArgs {
  const void* dh[RR_MAX_RANKS];
  const void* a[RR_MAX_RANKS];
  const void* u[RR_MAX_RANKS];
  uint32_t off[RR_MAX_RANKS + 1];
  uint32_t rows[RR_MAX_RANKS];
  int32_t p;
  const float* pre;        // NULL: a and u; else columns as those of `grad`
  int32_t pre32;           // a and u are float32
  void* grad;
  uint64_t ld;
  uint32_t tokens;
  // float16: the rows' scales (row_max), and of the hidden rows (row_exp; NULL: not needed)
  float* row_max;
  int32_t* row_exp;
  const void* x;
  uint32_t dim;
};

// Rows of x into aligned rows; float16: times a power of two (row_max, scale).
struct GatedRowsArgs {
  const void* x;
  void* out;
  uint64_t out_stride;
  const float* row_max;    // NULL: as they are
  const int32_t* row_exp;  // float16, riders: where the scale comes from (else from `scale`)
  int32_t* scale;
  uint32_t tokens, dim;
};

struct GatedJoinArgs {
  const float* acc;
  uint64_t split_stride;
  uint32_t acc_ld;
  const float* row_max;    // float16
  void* out;
  uint32_t tokens, dim, splits;
};

// dhidden += grad * weights over the columns of a piece.
struct GatedHiddenArgs {
  GatedShards sh;
  const void* grad;        // at the piece's first column
  uint64_t ld;
  uint64_t w_stride;
  float* acc;              // [splits][tokens][acc_ld] float32
  uint64_t split_stride;
  uint32_t acc_ld;         // dim in whole fours
  void* out;               // dhidden, where one product is all of it; else NULL
  const float* row_max;    // float16
  uint32_t tokens, dim;
  uint32_t c0, c1;         // columns
  uint32_t tiles_m, tiles_n, splits;
  int32_t add;
  // Short steps: the first `riders` workgroups copy kGatedRiderRows rows each,
  // which nothing in this launch reads.
  uint32_t riders;
  GatedRowsArgs copy;
};
constexpr uint32_t kGatedRiderRows = 8;

// dgate and dup = grad^T * x.
struct GatedWeightArgs {
  void* dgate[RR_MAX_RANKS];
  void* dup[RR_MAX_RANKS];
  uint32_t off[RR_MAX_RANKS + 1];
  uint32_t rows[RR_MAX_RANKS];
  int32_t p;
  const void* grad;
  uint64_t ld;
  const void* x;           // rows of x_stride bytes (float16: scaled)
  uint64_t x_stride;
  const int32_t* scale;    // float16
  uint32_t tokens, dim;
  uint32_t c0, c1;         // columns
  uint32_t tiles_m, tiles_n;
  // Short steps: workgroups [rider0, rider0 + riders) join dhidden, `join_cols`
  // of them a row; rider0: 0, or behind the tiles.
  uint32_t riders, rider0, join_cols;
  GatedJoinArgs join;
  // Few tiles: the tokens in `splits` parts, each with float32 sums [columns][acc_ld]
  // of its own, acc_stride floats apart (k_gated_weight_join); splits == 1: the results.
  float* acc;
  uint64_t acc_stride;
  uint32_t acc_ld;
  uint32_t splits;
};

struct GatedPackArgs {
  GatedShards sh;
  void* out;               // rows of features [f0, f1) of the gate, then of up
  uint64_t out_stride;
  uint32_t dim;
  uint32_t f0, f1;
  const void* x;  // with them: `tokens` rows of the hidden states, to x_out (0: none)
  void* x_out;
  uint32_t tokens;
};

hipError_t launch_gated(const GatedArgs& a, Kind k, GatedAct act, GatedMode m, GatedTile t, hipStream_t s);
hipError_t launch_gated_grad(const GatedGradArgs& a, Kind k, GatedAct act, hipStream_t s);
hipError_t launch_gated_hidden(const GatedHiddenArgs& a, Kind k, GatedTile t, hipStream_t s);
hipError_t launch_gated_weight(const GatedWeightArgs& a, Kind k, GatedTile t, hipStream_t s);
hipError_t launch_gated_pack(const GatedPackArgs& a, Kind k, hipStream_t s);
hipError_t launch_gated_rows(const GatedRowsArgs& a, Kind k, hipStream_t s);
hipError_t launch_gated_scale(const int32_t* row_exp, uint32_t tokens, int32_t* scale, hipStream_t s);
hipError_t launch_gated_join(const GatedJoinArgs& a, Kind k, hipStream_t s);
hipError_t launch_gated_weight_join(const GatedWeightArgs& a, Kind k, hipStream_t s);

// The matrix-product launchers of one element kind (one translation unit each).
#define RR_GATED_KIND(NAME)                                                                              \
  hipError_t launch_gated_##NAME(const GatedArgs& a, GatedAct act, GatedMode m, GatedTile t, hipStream_t s); \
  hipError_t launch_gated_hidden_##NAME(const GatedHiddenArgs& a, GatedTile t, hipStream_t s);           \
  hipError_t launch_gated_weight_##NAME(const GatedWeightArgs& a, GatedTile t, hipStream_t s);
RR_GATED_KIND(f32)
RR_GATED_KIND(bf16)
RR_GATED_KIND(f16)
#undef RR_GATED_KIND

// ---------------------------------------------------------------------------
// The plan of one call (rr_gated.cpp).
struct GatedPlan {
  GatedShards sh;          // gate and up unset
  uint32_t tokens, dim, dim_pad, esz;
  uint32_t acc_ld;         // floats of a row of sums: dim in whole fours
  uint32_t piece;          // padded features of a piece (all, unless the inputs are copied)
  uint64_t ld;             // columns of the gradients' matrix
  GatedTile forward_tile, hidden_tile, weight_tile;
  uint32_t splits;         // of dhidden
  uint32_t weight_splits;
  // workspace offsets in bytes
  uint64_t pack_x, pack_w, grad, pre, acc, weight_acc, xs, row_max, row_exp, scale, total;

  // dhidden is one product, written without sums of parts.
  bool direct() const { return splits == 1 && piece >= sh.off[sh.p]; }
};

// pack: the inputs are copied into aligned rows first; kept: the forward pass keeps its
// products, or the gradient is given them.  The sizes must be valid.
void plan_gated(GatedPlan& pl, int p, uint32_t tokens, uint32_t dim, uint32_t ffn, rr_dtype_t dt, bool grad, bool pack,
                bool kept);

// Where the columns [c0, c1) of a product go over from tiles of 256 to small ones (c1:
// nowhere); other: the product's other axis; steps: of K, 64 each.
enum class GatedUse : int { kForward, kForwardWide, kWeights };  // (wide: three matrices in or out)
uint32_t gated_tail(uint32_t c0, uint32_t c1, uint32_t other, uint32_t steps, GatedTile t, bool f32, GatedUse use);

// Up to so many tokens the small passes of the gradient (the copy of the hidden
// rows with float16's scale, the join of dhidden) ride on the products' launches,
// where those are of small tiles (96 x 768 x 2048 float16 step 60 -> 48 us).
// Longer ones copy and join so much that they want more workgroups a compute unit
// than the products' LDS leaves; the join of float32 and bfloat16 later than the rest (in a
// launch of its own / riding, us: 2000 x 768 x 2048 bfloat16 62 / 56, 1500 x 770 x 2050 float32
// 217 / 212, 3000 x 512 x 2048 72.2 / 71.9, 6000 x 512 x 1024 69.8 / 71.7; float16, 1500 x 1024 x
// 4096 105 / 107.6).
constexpr uint32_t kGatedRideTokens = 1024, kGatedJoinTokens = 4096;

constexpr uint32_t kGatedJoinMany = 8;  // splits from which 4 threads share a column of the join

constexpr GatedTile gated_small(bool f32) { return f32 ? GatedTile::k128x64 : GatedTile::k128x128; }

}  // namespace rr
