// rr_vocab.cpp -- plan of the vocabulary cross entropy: the padded vocabulary,
// its pieces, the tiles of the matrix products, and the workspace's layout.
// Host code only.
#include "rr_vocab.h"

#include <string.h>

#include <algorithm>

namespace rr {

namespace {

// The gradient of the logits of one piece of the vocabulary is kept at a time
// (storage type): a piece is as wide as fits here.
constexpr uint64_t kGradBytes = 1ull << 30;
// Copied weight rows of one piece (inputs whose rows are not 16-byte aligned).
constexpr uint64_t kPackBytes = 64ull << 20;
constexpr uint32_t kPieceUnit = 256;
constexpr uint32_t kUnits = 256;  // compute units

uint32_t ceil_div(uint64_t a, uint64_t b) { return static_cast<uint32_t>((a + b - 1) / b); }

}  // namespace

// A grid of large tiles, one on each compute unit, runs in rounds.  A last round
// that fills less than half of the units is given to small tiles, which spread
// it over all of them: as many whole tile columns as do not fit into the rounds
// before it, where they hold less than half a round.
uint32_t tail_start(uint32_t c0, uint32_t c1, uint32_t other_tiles, VocabTile t) {
  if (t != VocabTile::k256x256 || other_tiles == 0) return c1;
  const uint64_t tiles = static_cast<uint64_t>(ceil_div(c1 - c0, 256)) * other_tiles;
  const uint64_t full = tiles / kUnits * kUnits / other_tiles;  // tiles of this axis in full rounds
  const uint64_t moved = tiles - full * other_tiles;
  if (tiles < kUnits || moved == 0 || 2 * moved >= kUnits) return c1;
  return c0 + static_cast<uint32_t>(full) * 256;
}

void plan_vocab(VocabPlan& pl, int p, uint32_t tokens, uint32_t dim, uint32_t vocab, rr_dtype_t dt, bool grad,
                bool pack) {
  memset(&pl, 0, sizeof(pl));
  pl.tokens = tokens;
  pl.tokens_pad = ceil_div(tokens, kSlot) * kSlot;
  pl.dim = dim;
  pl.esz = dt == RR_FLOAT32 ? 4 : 2;
  const uint32_t epc = 16 / pl.esz;
  pl.dim_pad = ceil_div(dim, epc) * epc;
  pl.sh.p = p;
  pl.sh.vocab = vocab;
  uint32_t off = 0;
  for (int r = 0; r < p; ++r) {
    const uint32_t lo = static_cast<uint32_t>(static_cast<uint64_t>(r) * vocab / p);
    const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(r + 1) * vocab / p);
    pl.sh.first[r] = lo;
    pl.sh.rows[r] = hi - lo;
    pl.sh.off[r] = off;
    off += ceil_div(hi - lo, kSlot) * kSlot;
  }
  pl.sh.off[p] = off;

  const uint64_t row = static_cast<uint64_t>(pl.dim_pad) * pl.esz;
  uint64_t most = off;
  if (grad && pl.tokens_pad) most = std::min<uint64_t>(most, kGradBytes / (static_cast<uint64_t>(pl.tokens_pad) * pl.esz));
  if (pack) most = std::min<uint64_t>(most, kPackBytes / row);
  // a grid of at most 2^22 workgroups, and 32-bit offsets within a tile
  most = std::min<uint64_t>(most, 1u << 20);
  most = std::min<uint64_t>(most, (1ull << 22) / std::max(1u, ceil_div(tokens, 256)) * 256);
  if (most >= off) {
    pl.piece = off;
  } else {
    most = std::max<uint64_t>(most / kPieceUnit * kPieceUnit, kPieceUnit);
    pl.piece = ceil_div(ceil_div(off, ceil_div(off, most)), kPieceUnit) * kPieceUnit;
  }
  pl.pieces = ceil_div(off, pl.piece);

  // Tiles.  Up to 32 tokens take the narrow one.  Logits of up to 64 tokens, or of
  // so few 128 x 128 tiles that half of the units would idle, take 64 x 64 ones:
  // the weights are read by more units at once, and less of a tile is padding
  // (whole step, 128 x 128 / 64 x 64 tiles, us: 90 x 512 x 11000 (86 tiles) 49.7 / 45.4;
  // 128 x 4096 x 8000 (63) 142 / 125; 500 x 1024 x 2000 (64) 67.5 / 57.9; 128 x 2048 x
  // 24000 (188) 135 / 139; 50 x 512 x 120000 192 / 148; 60 x 1024 x 60000 145.1 / 144.6;
  // float32, 128 x 64 / 64 x 64: 250 x 1024 x 12000 (188) 263 / 236, 60 x 1024 x 60000
  // (469) 340 / 344).  The large tile reads least per
  // product, but only one workgroup fits on a compute unit, so nothing
  // overlaps its first loads and its output: it needs enough tiles for the
  // units, and enough steps of K in each.  Measured in bfloat16 on cold caches
  // (tokens x dim x vocabulary: large / small tile, us):
  //   logits, by the tiles: 1024 x 4096 x 32000 (500 tiles) 233 / 298; 256 x 4096
  //     x 32000 (125) 128 / 118; 512 x 768 x 50257 (394) 71 / 72;
  //   dhidden, by the steps over all tiles: 2048 x 768 x 50257 (18864) 416 / 435;
  //     4096 x 512 x 32000 (16000) 395 / 413; 512 x 768 x 50257 (4716) 174 / 162;
  //     1024 x 1024 x 8000 (2000) 102 / 71;
  //     (from 512 tokens on: the rule does not see how much of a large tile fewer
  //     tokens leave empty, and was not measured there);
  //   dweights, by the tokens: 2048 x 768 x 50257 422 / 435; 4096 x 512 x 32000 354 /
  //     398; 1024 x 4096 x 32000 613 / 587; 512 x 2048 x 16000 133 / 110.
  const uint32_t piece = pl.piece, steps = piece / kSlot;
  const uint64_t tt = ceil_div(tokens, 256), dd = ceil_div(dim, 256), vv = ceil_div(piece, 256);
  const auto pick = [&](bool large) { return large ? VocabTile::k256x256 : small_tile(pl.esz == 4); };
  if (tokens <= 32) {
    pl.logits_tile = pl.hidden_tile = VocabTile::k128x32;
  } else {
    const uint64_t tiles = static_cast<uint64_t>(ceil_div(piece, 128)) * ceil_div(tokens, 128);
    const bool f32 = pl.esz == 4;
    pl.logits_tile = pick(vv * tt >= kUnits);
    if (f32 ? tiles <= kUnits : tiles <= kUnits / 2 || tokens <= 64) pl.logits_tile = VocabTile::k64x64;
    pl.hidden_tile = pick(dd * tt * steps >= 32 * kUnits);
  }
  pl.weight_tile = pick(tokens >= 2048 && dd * vv >= kUnits * 3 / 4);
  // Few tiles of dhidden: K (the vocabulary) is split over one workgroup a unit
  // (two of float32's small ones), each with at least 4 steps.  (Two a unit in
  // bfloat16: 256 x 1024 x 16000 62 instead of 55 us, 96 x 768 x 50257 83 instead of
  // 78, 256 x 4096 x 32000 235 instead of 238.)
  const uint64_t htiles = static_cast<uint64_t>(ceil_div(dim, tile_m(pl.hidden_tile))) *
                          ceil_div(std::max(tokens, 1u), tile_n(pl.hidden_tile));
  const uint32_t want = pl.hidden_tile == VocabTile::k128x64 ? 2 * kUnits : kUnits;
  pl.splits = static_cast<uint32_t>(std::max<uint64_t>(std::min<uint64_t>(want / htiles, std::max(1u, steps / 4)), 1));

  for (uint32_t c0 = 0; c0 < off; c0 += pl.piece) {
    const uint32_t c1 = std::min(off, c0 + pl.piece);
    const uint32_t cm = tail_start(c0, c1, ceil_div(tokens, 256), pl.logits_tile);
    pl.tiles += ceil_div(cm - c0, tile_m(pl.logits_tile)) + ceil_div(c1 - cm, 128);
  }

  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  if (!grad) {
    pl.part = take(static_cast<uint64_t>(pl.tiles) * tokens * 8);
    pl.hit = take(static_cast<uint64_t>(tokens) * 4);
  } else {
    pl.xg = take(pl.tokens_pad * row);
    pl.grad = take(static_cast<uint64_t>(pl.tokens_pad) * piece * pl.esz);
    pl.acc = take(static_cast<uint64_t>(pl.splits) * tokens * dim * 4);
    pl.tcol = take(static_cast<uint64_t>(tokens) * 4);
    pl.lo = take(static_cast<uint64_t>(tokens) * 4);
    if (dt == RR_FLOAT16) pl.row_exp = take(static_cast<uint64_t>(tokens) * 4);
    pl.scale = take(4);
  }
  if (pack) {
    pl.pack_x = take(pl.tokens * row);
    pl.pack_w = take(piece * row);
  }
  pl.total = at;
}

}  // namespace rr
