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

uint32_t ceil_div(uint64_t a, uint64_t b) { return static_cast<uint32_t>((a + b - 1) / b); }

}  // namespace

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
  most = std::max<uint64_t>(most / kPieceUnit * kPieceUnit, kPieceUnit);
  pl.pieces = ceil_div(off, most);
  pl.piece = ceil_div(ceil_div(off, pl.pieces), kPieceUnit) * kPieceUnit;
  pl.pieces = ceil_div(off, pl.piece);

  // Tiles: the large tile reads least per product, where there are enough of
  // them for the 256 compute units; few tokens take the narrow one.
  const uint32_t piece = std::min(pl.piece, off);
  if (tokens <= 32) {
    pl.logits_tile = pl.hidden_tile = VocabTile::k128x32;
  } else {
    pl.logits_tile = static_cast<uint64_t>(ceil_div(piece, 256)) * ceil_div(tokens, 256) >= 256 ? VocabTile::k256x256
                                                                                                  : VocabTile::k128x128;
    pl.hidden_tile = static_cast<uint64_t>(ceil_div(dim, 256)) * ceil_div(tokens, 256) >= 64 ? VocabTile::k256x256
                                                                                              : VocabTile::k128x128;
  }
  pl.weight_tile = static_cast<uint64_t>(ceil_div(dim, 256)) * ceil_div(piece, 256) >= 256 ? VocabTile::k256x256
                                                                                            : VocabTile::k128x128;
  // Few tiles of dhidden: K (the vocabulary) is split over enough workgroups to
  // fill the chip, each with at least 4 steps.
  const uint64_t htiles = static_cast<uint64_t>(ceil_div(dim, tile_m(pl.hidden_tile))) *
                          ceil_div(std::max(tokens, 1u), tile_n(pl.hidden_tile));
  const uint32_t want = pl.hidden_tile == VocabTile::k256x256 ? 256 : pl.hidden_tile == VocabTile::k128x128 ? 512 : 1024;
  const uint32_t steps = piece / kSlot;
  uint64_t splits = std::min<uint64_t>(ceil_div(want, htiles), std::max(1u, steps / 4));
  pl.splits = static_cast<uint32_t>(std::max<uint64_t>(splits, 1));

  for (uint32_t i = 0; i < pl.pieces; ++i) {
    const uint32_t c0 = i * pl.piece, c1 = std::min(off, c0 + pl.piece);
    pl.tiles += ceil_div(c1 - c0, tile_m(pl.logits_tile));
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
    pl.scale = take(4);
  }
  if (pack) {
    pl.pack_x = take(pl.tokens * row);
    pl.pack_w = take(piece * row);
  }
  pl.total = at;
}

}  // namespace rr
