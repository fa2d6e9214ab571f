// rr_gated.cpp -- plan of the gated column-parallel projections: padded
// features, pieces, the tiles of the matrix products, and the workspace's
// layout.  Host code only.
#include "rr_gated.h"

#include <string.h>

#include <algorithm>

namespace rr {

namespace {

constexpr uint64_t kPackBytes = 64ull << 20;  // copied weight rows of one piece
constexpr uint32_t kUnits = 256;              // compute units
constexpr uint32_t kFewTokens = 64, kFewTokensCopied = 128;

uint32_t ceil_div(uint64_t a, uint64_t b) { return static_cast<uint32_t>((a + b - 1) / b); }

// What a product of 16-bit types over m x n and `steps` steps of 64 takes in tiles t, in
// 0.01 us: rounds of tiles over the chip, each with its first loads and output and its
// steps.  256 x 256 and 256 x 192 tiles fill a compute unit alone, 128 x 128 ones in pairs,
// one's output under the other's products.  wide: the output is three matrices of the
// forward pass, or two and the read of a third.
// Fitted to the forward pass (tokens x dim x ffn: 128 x 128 / 256 x 192 / 256 x 256, us): 1500 x 1024
// x 4096 29 / 27 / 32; 768 x 2048 x 8192 53 / 48 / 54; 1500 x 4096 x 4096 97 / 86 / 91; 1000 x 4096 x
// 4096 64 / 74 / 83; 2048 x 2048 x 4096 66 / 82 / 60; 8192 x 256 x 1024 15 / 23 / 18; 4096 x 1024 x 4096
// 71 / 75 / 68; 2048 x 4096 x 11008 352 / 341 / 316; with both products kept in float32: 8192 x 1024
// x 4096 177 / 206 / 212; 8192 x 768 x 2048 78 / 91 / 94; 8192 x 2048 x 4096 288 / 311 / 299; 8192 x 4096
// x 4096 523 / 523 / 488; 1500 x 1024 x 4096 41 / 39 / 51.  It misses 512 x 4096 x 11008, 116 / 148 / 104.
// (Weights still in the caches.  From memory 128 x 128 tiles, which read most, lose up to a
// tenth; over 143 drawn shapes what is chosen then takes 0.5 % more than the quickest, at worst 13 %:
// 512 x 4096 x 11008, and 8192 x 2048 x 4096 kept, 320 / 302 / 281.  A margin for the larger tiles
// gains at these and loses elsewhere.)
uint64_t round_time(uint64_t m, uint64_t n, uint32_t steps, GatedTile t, bool wide) {
  const uint64_t tiles = static_cast<uint64_t>(ceil_div(m, tile_m(t))) * ceil_div(n, tile_n(t));
  switch (t) {
    case GatedTile::k256x256: return (tiles + kUnits - 1) / kUnits * ((wide ? 2450 : 1050) + 153 * steps);
    case GatedTile::k256x192: return (tiles + kUnits - 1) / kUnits * ((wide ? 1600 : 800) + 120 * steps);
    default: {
      const uint64_t rest = tiles % (2 * kUnits), ends = wide ? 690 : 350;
      return tiles / (2 * kUnits) * (ends + 93 * steps) +
             (rest == 0 ? 0 : ends + (rest <= kUnits ? 60 : 93) * steps);
    }
  }
}

// The same for float32's dhidden in 128 x 64 tiles and `parts` along K, with the parts'
// sums, written and read.
uint64_t parts_time(uint64_t tiles, uint64_t parts, uint32_t steps, uint64_t outputs) {
  const uint64_t n = tiles * parts, rest = n % (2 * kUnits);
  const uint32_t each = ceil_div(steps, parts), two = 300 + 340 * each, one = 300 + 250 * each;
  return n / (2 * kUnits) * two + (rest == 0 ? 0 : rest <= kUnits ? one : two) + parts * outputs / 7500;
}

// The quickest tiles of a product whose first axis are columns.
GatedTile quickest(uint32_t columns, uint32_t other, uint32_t steps, GatedUse use) {
  const bool wide = use == GatedUse::kForwardWide;
  const uint32_t at = gated_tail(0, columns, other, steps, GatedTile::k256x256, false, use);
  uint64_t best = round_time(at, other, steps, GatedTile::k256x256, wide);
  if (at < columns) best += round_time(columns - at, other, steps, GatedTile::k128x128, wide);
  GatedTile tile = GatedTile::k256x256;
  for (const GatedTile t : {GatedTile::k256x192, GatedTile::k128x128}) {
    if (use == GatedUse::kWeights && t == GatedTile::k256x192) continue;
    const uint64_t time = round_time(columns, other, steps, t, wide);
    if (time < best) best = time, tile = t;
  }
  return tile;
}

}  // namespace

// A grid of large tiles, one on each compute unit, runs in rounds.  What does not fill a
// last round goes to small tiles, in 16-bit types where round_time says that they take less
// than 7/10 of it (2000 x 4096 x 9000, the last 56 of 568 tiles: 275 -> 259 us; the weights of
// 5000 x 2048 x 5000, 64 of 320: 258 -> 244; 2048 x 4096 x 11008, 176 of 688 tiles as 242 of 256 x
// 192, 8/10 of the round by the model: 318 -> 325), in float32 where it is less than half a round.
uint32_t gated_tail(uint32_t c0, uint32_t c1, uint32_t other, uint32_t steps, GatedTile t, bool f32, GatedUse use) {
  const uint64_t across = ceil_div(other, 256), tiles = ceil_div(c1 - c0, 256) * across;
  if (t != GatedTile::k256x256 || tiles < kUnits) return c1;
  const uint64_t full = tiles / kUnits * kUnits / across;  // tiles of the columns in full rounds
  const uint64_t moved = tiles - full * across;
  if (full == 0 || moved == 0) return c1;
  const uint32_t at = c0 + static_cast<uint32_t>(full) * 256;
  if (f32) return 2 * moved < kUnits ? at : c1;
  const bool wide = use == GatedUse::kForwardWide;
  return 10 * round_time(c1 - at, other, steps, gated_small(false), wide) <
                 7 * round_time(c1 - at, other, steps, t, wide)
             ? at
             : c1;
}

void plan_gated(GatedPlan& pl, int p, uint32_t tokens, uint32_t dim, uint32_t ffn, rr_dtype_t dt, bool grad,
                bool pack, bool kept) {
  memset(&pl, 0, sizeof(pl));
  pl.tokens = tokens;
  pl.dim = dim;
  pl.esz = dt == RR_FLOAT32 ? 4 : 2;
  const uint32_t epc = 16 / pl.esz;
  pl.dim_pad = ceil_div(dim, epc) * epc;
  pl.acc_ld = ceil_div(dim, 4) * 4;
  pl.sh.p = p;
  uint32_t off = 0;
  for (int r = 0; r < p; ++r) {
    const uint32_t lo = static_cast<uint32_t>(static_cast<uint64_t>(r) * ffn / p);
    const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(r + 1) * ffn / p);
    pl.sh.rows[r] = hi - lo;
    pl.sh.off[r] = off;
    off += ceil_div(hi - lo, kFeat) * kFeat;
  }
  pl.sh.off[p] = off;
  pl.ld = 2ull * off;

  const bool f32 = pl.esz == 4;
  const uint64_t row = static_cast<uint64_t>(pl.dim_pad) * pl.esz;
  uint64_t fits = off;
  if (pack) fits = std::max<uint64_t>(kPackBytes / (2 * row) / 128 * 128, 128);
  pl.piece = fits >= off ? off : ceil_div(ceil_div(off, ceil_div(off, fits)), 128) * 128;
  // Columns of one launch of the forward pass and of dhidden: the tiles are chosen for these
  // (for all columns: 864 x 2899 x 14336 in float32, six pieces, 4350 us instead of 1570).
  const uint32_t columns = 2 * pl.piece;

  const uint64_t tt = ceil_div(tokens, 256), dd = ceil_div(dim, 256);
  const auto pick = [&](bool large) { return large ? GatedTile::k256x256 : gated_small(f32); };
  // Forward tiles.  Few tokens: kFew up to 64, and where the rows would have to be
  // copied, which it reads as they lie, up to 128; few tiles: the small ones, so that
  // more units take part (float32, whose products take longer than its loads at any of
  // these sizes, up to more tiles); else by round_time, in float32 the large one where there
  // is one for every unit.  Measured (tokens x dim x ffn: kFew / 64 x 64 / 128 x 128, in
  // float32 128 x 64, us): 48 x 4096 x 11008 47 / 51 / 52; 64 x 4096 x 11008 50.5 / 51.5 / 51.7;
  // 96 x 768 x 2048 10.9 / 9.0 / 11.6; 96 x 4096 x 11008 (172 tiles of 128 x 128) 74 / 58 / 54; 128
  // x 1024 x 4096 (64) 13.0 / 10.6 / 13.7; 500 x 768 x 2048 (128) 11.3 / 12.0; 512 x 1024 x 4096
  // (256) 20.9 / 15.6; float32: 64 x 770 x 2050 17.6 / 33 / 46, 128 x 770 x 2050 32 / 35 / 47, 700 x
  // 768 x 2048 (352) - / 43 / 54, 333 x 4096 x 4096 (768) - / 195 / 251, 1000 x 1024 x 4096
  // (1024) - / 142 / 138.
  const uint64_t mid = static_cast<uint64_t>(ceil_div(columns, 128)) * ceil_div(tokens, tile_n(gated_small(f32)));
  if (tokens <= (pack ? kFewTokensCopied : kFewTokens)) {
    pl.forward_tile = GatedTile::kFew;
  } else if (mid <= (f32 ? 3 * kUnits : kUnits / 2)) {
    pl.forward_tile = GatedTile::k64x64;
  } else if (f32) {
    pl.forward_tile = pick(ceil_div(columns, 256) * tt >= kUnits);
  } else {
    // (the gradient's products again, with dh read, are as wide as those that are kept)
    pl.forward_tile = quickest(columns, tokens, ceil_div(dim, 64),
                               kept || grad ? GatedUse::kForwardWide : GatedUse::kForward);
  }
  const uint32_t steps = columns / kFeat;
  // dhidden, by the steps of K over all tiles (256 x 256 / 128 x 128, with the activation's
  // gradient, us): 2048 x 4096 x 11008 (172 steps a workgroup) 391 / 446, 512 x 4096 x 11008
  // (43) 125 / 139, 4096 x 1024 x 4096 (32) 129 / 129, 8192 x 1024 x 2048 (32) 131 / 112.  The
  // weights' gradients by round_time, in float32 by the tokens and the tiles: 2048 x 4096 x 11008
  // 409 / 442, 512 x 4096 x 11008 133 / 128, 8192 x 1024 x 2048 (64 tiles of 256 x 256) 187 / 116.
  pl.hidden_tile = tokens <= 32 ? GatedTile::k128x32 : pick(dd * tt * steps >= 40 * kUnits);
  pl.weight_tile = f32 ? pick(tokens >= 2048 && dd * ceil_div(pl.ld, 256) >= kUnits * 3 / 4)
                       : quickest(static_cast<uint32_t>(pl.ld), dim, ceil_div(tokens, 64), GatedUse::kWeights);

  const uint64_t htiles = static_cast<uint64_t>(ceil_div(dim, tile_m(pl.hidden_tile))) *
                          ceil_div(std::max(tokens, 1u), tile_n(pl.hidden_tile));
  // dhidden's parts along K.  One workgroup a compute unit; two, where that would leave a
  // quarter of the units without one.  Float32's small tiles: what parts_time finds quickest
  // (two workgroups a unit / that, us: 1500 x 1024 x 4096 283 / 232, 333 x 4096 x 4096 268 / 215; 16-bit
  // types by such a model: 1000 x 2048 x 8192 108 / 101, but 4096 x 1024 x 4096 117 / 124).
  const uint64_t most = std::max<uint64_t>(steps / 4, 1);
  uint32_t want = kUnits;
  if (pl.hidden_tile != GatedTile::k256x256 && want / htiles * htiles <= kUnits * 3 / 4) want = 2 * kUnits;
  pl.splits = static_cast<uint32_t>(std::max<uint64_t>(std::min<uint64_t>(want / htiles, most), 1));
  if (pl.hidden_tile == GatedTile::k128x64) {
    uint64_t best = ~0ull;
    for (uint64_t n = 1; n <= std::min<uint64_t>(most, 16 * kUnits / htiles + 1); ++n) {
      const uint64_t t = parts_time(htiles, n, steps, static_cast<uint64_t>(tokens) * dim);
      if (t < best) best = t, pl.splits = static_cast<uint32_t>(n);
    }
  }

  // Few tiles of the weights' gradients: the tokens in parts, of eight steps or more, so
  // that there is a workgroup for each unit, and a launch that adds the parts; 16-bit types
  // from 24 steps on (tokens x dim x ffn, whole gradient without dhidden, in one part / in
  // parts, us: 8192 x 64 x 128 67 / 14, 8192 x 512 x 1024 80 / 49, 2048 x 256 x 512 22 / 18, 1024 x
  // 256 x 512 14.2 / 14.5, in float32 42 / 29).
  const uint64_t wtiles = static_cast<uint64_t>(ceil_div(dim, tile_m(pl.weight_tile))) *
                          ceil_div(pl.ld, tile_n(pl.weight_tile));
  const uint32_t token_steps = ceil_div(tokens, 64);
  pl.weight_splits = 1;
  if (pl.weight_tile != GatedTile::k256x256 && (f32 || token_steps >= 24))
    pl.weight_splits = static_cast<uint32_t>(
        std::max<uint64_t>(std::min<uint64_t>(kUnits / wtiles, token_steps / 8), 1));

  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  if (grad) {
    pl.grad = take(tokens * pl.ld * pl.esz);
    if (!pl.direct()) pl.acc = take(static_cast<uint64_t>(pl.splits) * tokens * pl.acc_ld * 4);
    if (pl.weight_splits > 1) pl.weight_acc = take(pl.weight_splits * pl.ld * pl.acc_ld * 4);
    if (dt == RR_FLOAT16) {
      if (!kept) pl.pre = take(tokens * pl.ld * 4);
      pl.xs = take(tokens * row);
      pl.row_max = take(static_cast<uint64_t>(tokens) * 4);
      pl.row_exp = take(static_cast<uint64_t>(tokens) * 4);
      pl.scale = take(4);
    }
  }
  if (pack && (grad || pl.forward_tile != GatedTile::kFew)) {
    pl.pack_x = take(tokens * row);
    pl.pack_w = take(2ull * pl.piece * row);
  }
  pl.total = at;
}

}  // namespace rr
