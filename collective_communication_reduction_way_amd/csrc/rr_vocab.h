// rr_vocab.h -- plan and argument blocks of the vocabulary-parallel softmax
// cross entropy (internal to librr.so).
//
// The vocabulary's V rows are cut over the p virtual ranks at the chunk bounds
// floor(r*V/p).  The kernels work in a "padded vocabulary": every shard's rows
// rounded up to a multiple of kSlot, the shards laid end to end, so that a
// slot of kSlot columns never crosses a shard and a K step over the
// vocabulary reads one shard.  Columns that pad a slot have no logit.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "rr.h"
#include "rr_kernels.h"

namespace rr {

constexpr uint32_t kSlot = 64;
constexpr uint32_t kMasked = 0xFFFFFFFFu;  // "padded column" of a masked token's target

struct VocabShards {
  const void* w[RR_MAX_RANKS];       // row 0 of each shard's [rows, dim] matrix
  uint32_t off[RR_MAX_RANKS + 1];    // first padded column of each shard; off[p] = all padded columns
  uint32_t rows[RR_MAX_RANKS];       // the shard's own rows
  uint32_t first[RR_MAX_RANKS];      // its first row in the vocabulary
  int32_t p;
  uint32_t vocab;
};

// Tile of the matrix products: (columns of the M axis) x (columns of the N axis).
// k128x64: float32 only; k64x64: logits only.
enum class VocabTile : int { k256x256 = 0, k128x128 = 1, k128x32 = 2, k128x64 = 3, k64x64 = 4 };
constexpr uint32_t tile_m(VocabTile t) {
  return t == VocabTile::k256x256 ? 256 : t == VocabTile::k64x64 ? 64 : 128;
}
constexpr uint32_t tile_n(VocabTile t) {
  switch (t) {
    case VocabTile::k256x256: return 256;
    case VocabTile::k128x128: return 128;
    case VocabTile::k128x32: return 32;
    default: return 64;
  }
}

// Logits of a piece [c0, c1) of the padded vocabulary.  Forward: the running
// maximum and sum of exponentials of every M tile and token, and the target's
// logit.  Gradient: the gradient of the logits in the storage type.
struct LogitArgs {
  VocabShards sh;
  const void* x;          // [tokens, dim] rows of x_stride bytes
  uint64_t x_stride;
  uint64_t w_stride;      // bytes between rows of a shard
  const void* targets;
  const float* lse;       // gradient
  const float* grad_loss; // gradient
  float* part;            // forward: [tile][tokens][2] maximum and sum
  float* hit;             // forward: the target's logit
  void* grad;             // gradient: [tokens rounded up to kSlot][ld] in the storage type
  uint32_t* tcol;         // gradient: the targets' padded columns (kMasked: none)
  float* lo;              // gradient, 16-bit types: what rounding took from the target's entry
  uint64_t ld;
  uint32_t tokens;
  uint32_t grad_rows;     // gradient: rows of `grad`, zeros from `tokens` on
  uint32_t kbytes;        // dim * element size, a multiple of 16
  uint32_t c0, c1;
  uint32_t tile0;         // first forward tile of this piece in `part`
  uint32_t tiles_m, tiles_n;
  int32_t target_bytes;   // 4 or 8
  // Gradient, short steps: the first `riders` workgroups copy kRiderRows rows
  // each into xg (PackRowsArgs with unit = 16) and write tcol and, in float16,
  // scale, which nothing in this launch reads.
  uint32_t riders;
  void* xg;
  const int32_t* row_exp; // float16: of k_row_exponent; NULL: the rows are not scaled
  int32_t* scale;
};
constexpr uint32_t kRiderRows = 8;

// dhidden += grad * W over a piece: accumulators [split][tokens][dim] float32.
struct HiddenGradArgs {
  VocabShards sh;
  const void* grad;
  uint64_t ld;
  uint64_t w_stride;
  float* acc;
  uint64_t split_stride;  // floats between the splits' accumulators
  uint32_t tokens, dim;
  uint32_t grad_rows;     // rows of `grad`
  uint32_t c0, c1;
  uint32_t tiles_m, tiles_n, splits;
  int32_t add;            // 1: add to what the accumulators hold (pieces after the first)
  void* out;              // dhidden, where one product is all of it (rows 16-byte aligned); else NULL
  const uint32_t* tcol;   // with out: as in LogitArgs
  const float* lo;
  const float* grad_loss;
};

// dhidden from the sums of its splits: 4 threads share a column's where there
// are kJoinMany or more.
constexpr uint32_t kJoinMany = 8;
struct JoinPart {
  const float* acc;
  uint64_t split_stride;
  const float* grad_loss; // float16: for the row's scale; else NULL
  const uint32_t* tcol;
  const float* lo;        // 16-bit types
  void* out;
  uint32_t tokens, dim, splits;
  int32_t vec;            // 1: rows of the weights and of dhidden are 8-byte aligned
};

// dweights of a piece = grad^T * xg (xg: the hidden rows that count).
struct WeightGradArgs {
  VocabShards sh;
  void* dw[RR_MAX_RANKS];
  const void* grad;
  uint64_t ld;
  const void* xg;         // [tokens rounded up to kSlot][xg_stride bytes]
  uint64_t xg_stride;
  const int32_t* scale;   // float16: m of the tokens (token_exponent), on the device
  const uint32_t* tcol;   // as in LogitArgs
  const float* lo;
  uint32_t tokens;
  uint32_t rows;          // K: tokens rounded up to kSlot
  uint32_t dim;
  uint32_t c0, c1;
  uint32_t tiles_m, tiles_n;
  int32_t vec;            // 1: rows of dweights are 16-byte aligned
  // Short steps: workgroups [rider0, rider0 + riders) join dhidden, `join_cols`
  // of them a row (dim a multiple of 4); rider0: 0, or behind the tiles.
  uint32_t riders, rider0, join_cols;
  JoinPart join;
};

// Copies rows of `dim` elements into rows of out_stride bytes, zero-filled:
// the hidden rows (masked rows become zero when targets is given; float16
// rows are scaled by a power of two, see token_exponent).
struct PackRowsArgs {
  VocabShards sh;
  const void* x;
  void* out;
  const void* targets;    // NULL: every row counts
  const float* grad_loss; // NULL: no scaling
  const int32_t* scale;
  uint32_t* tcol;         // NULL, or the targets' padded columns are written here
  uint64_t out_stride;    // bytes
  uint32_t unit;          // bytes (16, 8, 4 or 2) that x and its rows are aligned to
  uint32_t tokens, rows;  // rows: written rows, zero from `tokens` on
  uint32_t dim;
  int32_t target_bytes;
};

// float16: every token's e + a (token_exponent), kNoExponent where its row counts
// for nothing.
struct RowExponentArgs {
  const void* x;
  const float* grad_loss;
  const void* targets;
  int32_t* out;
  uint32_t unit;          // as in PackRowsArgs
  uint32_t tokens, dim, vocab;
  int32_t target_bytes;
};

struct PackWeightArgs {
  VocabShards sh;
  void* out;              // row i = padded column c0 + i
  uint64_t out_stride;
  uint32_t unit;          // as in PackRowsArgs, of all shards
  uint32_t dim;
  uint32_t c0, c1;
};

struct LossArgs {
  const float* part;
  const float* hit;
  const void* targets;
  float* loss;
  float* lse;
  uint32_t tokens, tiles, vocab;
  int32_t target_bytes;
};

struct JoinArgs : JoinPart {
  VocabShards sh;         // the caller's weights
};

hipError_t launch_logits(const LogitArgs& a, Kind k, VocabTile t, bool grad, hipStream_t s);
hipError_t launch_hidden_grad(const HiddenGradArgs& a, Kind k, VocabTile t, hipStream_t s);
hipError_t launch_weight_grad(const WeightGradArgs& a, Kind k, VocabTile t, hipStream_t s);
hipError_t launch_pack_rows(const PackRowsArgs& a, Kind k, hipStream_t s);
hipError_t launch_pack_weight(const PackWeightArgs& a, Kind k, hipStream_t s);
hipError_t launch_loss(const LossArgs& a, hipStream_t s);
hipError_t launch_row_exponent(const RowExponentArgs& a, hipStream_t s);
hipError_t launch_grad_scale(const int32_t* row_exp, uint32_t tokens, int32_t* scale, hipStream_t s);
hipError_t launch_join(const JoinArgs& a, Kind k, hipStream_t s);

// The matrix-product launchers of one element kind (one translation unit each).
#define RR_VOCAB_KIND(NAME)                                                                    \
  hipError_t launch_logits_##NAME(const LogitArgs& a, VocabTile t, bool grad, hipStream_t s); \
  hipError_t launch_hidden_grad_##NAME(const HiddenGradArgs& a, VocabTile t, hipStream_t s);  \
  hipError_t launch_weight_grad_##NAME(const WeightGradArgs& a, VocabTile t, hipStream_t s);
RR_VOCAB_KIND(f32)
RR_VOCAB_KIND(bf16)
RR_VOCAB_KIND(f16)
#undef RR_VOCAB_KIND

// ---------------------------------------------------------------------------
// The plan of one call (rr_vocab.cpp): pieces, tiles, and the workspace's layout.
struct VocabPlan {
  VocabShards sh;         // w unset
  uint32_t tokens, tokens_pad, dim, dim_pad;
  uint32_t esz;
  uint32_t piece;         // padded columns of a piece
  uint32_t pieces;
  VocabTile logits_tile, hidden_tile, weight_tile;
  uint32_t splits;
  uint32_t tiles;         // forward M tiles over all pieces
  // workspace offsets in bytes
  uint64_t part, hit, pack_x, pack_w, xg, grad, acc, tcol, lo, row_exp, scale, total;
};

// The tile where there is too little work for the large one.
constexpr VocabTile small_tile(bool f32) { return f32 ? VocabTile::k128x64 : VocabTile::k128x128; }

// Up to so many tokens the small passes of the gradient (the copy of the hidden
// rows with float16's scale, the join of dhidden) ride on the products' launches,
// where those are of small tiles and read their inputs in place: three launches
// less, about 4 us each (96 x 768 x 50257 float16 step 123.9 -> 113.5 us, 20 x 256 x
// 4000 52 -> 44; 1024 x 2048 x 4000 float16 128 -> 119; since then float16 has a
// launch more for the rows' exponents, 3 us).  Longer ones copy and join
// so much that they want more workgroups a compute unit than the products' LDS
// leaves.
constexpr uint32_t kRideTokens = 1024;

// Where the columns [c0, c1) of a product go over from tiles `t` to small tiles
// (c1: nowhere); other_tiles: the 256-wide tiles of the product's other axis.
uint32_t tail_start(uint32_t c0, uint32_t c1, uint32_t other_tiles, VocabTile t);

// pack: the inputs are copied into aligned rows first.  The sizes must be valid.
void plan_vocab(VocabPlan& pl, int p, uint32_t tokens, uint32_t dim, uint32_t vocab, rr_dtype_t dt, bool grad,
                bool pack);

}  // namespace rr
