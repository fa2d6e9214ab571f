// rr_block.cpp -- C entry points of what stands in front of the row-parallel
// product of a tensor-parallel block: the norm over the ranks' rows, and the
// gated column-parallel projections.
// Checks of arguments, plans and launches; host code only.
#include <math.h>
#include <string.h>

#include "rr_gated.h"
#include "rr_host.h"
#include "rr_norm.h"

using namespace rr::host;
using rr::Kind;

namespace {

constexpr uint64_t kMaxNormRows = (1ull << 31) - 1;  // of all ranks: 32-bit row numbers

rr_status_t check_norm_shape(int p, size_t rows, size_t dim, rr_dtype_t dtype) {
  rr_status_t st;
  if ((st = check_p(p)) || (st = check_float_dtype(dtype, "the layer norm"))) return st;
  if (dim < 1 || dim > rr::kNormDim)
    return fail(RR_ERROR_INVALID_ARGUMENT, "dim=%zu outside [1, %u]", dim, rr::kNormDim);
  if (rows > kMaxNormRows / static_cast<uint64_t>(p))
    return fail(RR_ERROR_INVALID_ARGUMENT, "rows=%zu of %d ranks exceed 2^31 - 1", rows, p);
  return RR_SUCCESS;
}

// p buffers of one kind, added to `ranges`.
rr_status_t check_bufs(const void* const* bufs, const char* what, int p, size_t esz, uint64_t bytes,
                       std::vector<Range>& ranges) {
  if (!bufs) return fail(RR_ERROR_INVALID_ARGUMENT, "%s is NULL", what);
  for (int r = 0; r < p; ++r) {
    const rr_status_t st = check_buf(bufs[r], esz, what, r);
    if (st) return st;
    ranges.push_back(range_of(bufs[r], bytes, r));
  }
  return RR_SUCCESS;
}

rr_status_t check_one(const void* buf, const char* what, size_t esz, uint64_t bytes, int id,
                      std::vector<Range>& ranges) {
  const rr_status_t st = check_buf(buf, esz, what, 0);
  if (st) return st;
  ranges.push_back(range_of(buf, bytes, id));
  return RR_SUCCESS;
}

// An output may be an input of the same rank.
bool in_place(const Range& o, const Range& in) {
  return o.rank >= 0 && o.rank == in.rank && o.lo == in.lo && o.hi == in.hi;
}

rr_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return RR_SUCCESS;
  if (!workspace) return fail(RR_ERROR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned16(workspace)) return fail(RR_ERROR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
  if (have < need)
    return fail(RR_ERROR_INVALID_ARGUMENT, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  return RR_SUCCESS;
}

rr_status_t norm_body(const void* const* sendbufs, const void* weight, const void* bias, void* const* recvbufs,
                      float* mean, float* rstd, int p, size_t rows, size_t dim, double eps, int center,
                      rr_dtype_t dtype, rr_stream_t stream) {
  rr_status_t st;
  if ((st = check_norm_shape(p, rows, dim, dtype))) return st;
  if (!(eps >= 0) || !(static_cast<float>(eps) < INFINITY))
    return fail(RR_ERROR_INVALID_ARGUMENT, "eps=%g is not a finite number from 0 on", eps);
  if (mean && !center) return fail(RR_ERROR_INVALID_ARGUMENT, "a norm that is not centred has no mean");
  if (rows == 0) return ok();
  const size_t esz = rr::elem_size(dtype);
  const uint64_t bytes = static_cast<uint64_t>(rows) * dim * esz, total = static_cast<uint64_t>(rows) * p;
  std::vector<Range> ins, outs;
  if ((st = check_bufs(sendbufs, "sendbufs", p, esz, bytes, ins)) ||
      (st = check_bufs(recvbufs, "recvbufs", p, esz, bytes, outs)))
    return st;
  if (weight && (st = check_one(weight, "weight", esz, dim * esz, -1, ins))) return st;
  if (bias && (st = check_one(bias, "bias", esz, dim * esz, -2, ins))) return st;
  if (mean && (st = check_one(mean, "mean", 4, total * 4, -3, outs))) return st;
  if (rstd && (st = check_one(rstd, "rstd", 4, total * 4, -4, outs))) return st;
  if ((st = check_aliasing_sorted(outs, ins, in_place))) return st;
  rr::NormArgs a;
  for (int r = 0; r < p; ++r) {
    a.in[r] = sendbufs[r];
    a.out[r] = recvbufs[r];
  }
  a.weight = weight;
  a.bias = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = static_cast<uint32_t>(rows);
  a.total = static_cast<uint32_t>(total);
  a.dim = static_cast<uint32_t>(dim);
  a.eps = static_cast<float>(eps);
  // A lane's sum is of 32 squares at most; scaled by 2^-14 the row's sum fits float32 where
  // its mean does.  What that loses, below 2^-112 a lane, is nothing beside an eps of 2^-70.
  a.fit = eps >= 0x1p-70 ? 0x1p-14f : 1.f;
  a.back = 1.f / a.fit;
  a.center = center ? 1 : 0;
  if (log_launches()) fprintf(stderr, "[rr] layer_norm: p=%d rows=%zu dim=%zu center=%d\n", p, rows, dim, a.center);
  const hipError_t e = rr::launch_norm(a, kind_of(dtype), reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "layer_norm");
  return ok();
}

rr_status_t norm_grad_body(const void* const* grad_outs, const void* const* sendbufs, const void* weight,
                           const float* mean, const float* rstd, const void* const* residuals, void* const* grad_ins,
                           void* dweight, void* dbias, int p, size_t rows, size_t dim, int center, rr_dtype_t dtype,
                           void* workspace, size_t workspace_bytes, rr_stream_t stream) {
  rr_status_t st;
  if ((st = check_norm_shape(p, rows, dim, dtype))) return st;
  if (!grad_ins && !dweight && !dbias)
    return fail(RR_ERROR_INVALID_ARGUMENT, "grad_ins, dweight and dbias are all NULL");
  if (residuals && !grad_ins) return fail(RR_ERROR_INVALID_ARGUMENT, "residuals without grad_ins");
  if (mean && !center) return fail(RR_ERROR_INVALID_ARGUMENT, "a norm that is not centred has no mean");
  const size_t esz = rr::elem_size(dtype);
  const uint64_t bytes = static_cast<uint64_t>(rows) * dim * esz, total = static_cast<uint64_t>(rows) * p;
  std::vector<Range> ins, outs;
  if (rows > 0) {
    if ((st = check_bufs(grad_outs, "grad_outs", p, esz, bytes, ins)) ||
        (st = check_bufs(sendbufs, "sendbufs", p, esz, bytes, ins)) ||
        (st = check_one(rstd, "rstd", 4, total * 4, -1, ins)) ||
        (center && (st = check_one(mean, "mean", 4, total * 4, -2, ins))) ||
        (residuals && (st = check_bufs(residuals, "residuals", p, esz, bytes, ins))) ||
        (grad_ins && (st = check_bufs(grad_ins, "grad_ins", p, esz, bytes, outs))))
      return st;
  }
  if (weight && (st = check_one(weight, "weight", esz, dim * esz, -3, ins))) return st;
  if (dweight && (st = check_one(dweight, "dweight", esz, dim * esz, -4, outs))) return st;
  if (dbias && (st = check_one(dbias, "dbias", esz, dim * esz, -5, outs))) return st;
  const bool sums = dweight || dbias;
  const Kind k = kind_of(dtype);
  const size_t need = sums ? rr_layer_norm_grad_workspace_size(p, rows, dim, dtype) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if (need) outs.push_back(range_of(workspace, workspace_bytes, -6));
  if ((st = check_aliasing_sorted(outs, ins, in_place))) return st;
  if (rows == 0 && !sums) return ok();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  rr::NormGradArgs a;
  memset(&a, 0, sizeof(a));
  if (rows > 0) {
    for (int r = 0; r < p; ++r) {
      a.dy[r] = grad_outs[r];
      a.x[r] = sendbufs[r];
      a.res[r] = residuals ? residuals[r] : nullptr;
      a.dx[r] = grad_ins ? grad_ins[r] : nullptr;
    }
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows = static_cast<uint32_t>(rows);
    a.total = static_cast<uint32_t>(total);
    a.dim = static_cast<uint32_t>(dim);
    a.center = center ? 1 : 0;
    a.has_dx = grad_ins ? 1 : 0;
    a.has_res = residuals ? 1 : 0;
    if (log_launches())
      fprintf(stderr, "[rr] layer_norm_grad: p=%d rows=%zu dim=%zu center=%d parts=%u\n", p, rows, dim, a.center,
              rr::norm_grad_grid(a.total, a.dim, k));
    const hipError_t e = rr::launch_norm_grad(a, k, s);
    if (e != hipSuccess) return hip_fail(e, "layer_norm_grad");
  }
  if (sums) {
    rr::NormJoinArgs j;
    j.part = static_cast<const float*>(workspace);
    j.dweight = dweight;
    j.dbias = dbias;
    j.parts = rr::norm_grad_grid(static_cast<uint32_t>(total), static_cast<uint32_t>(dim), k);
    j.dim = static_cast<uint32_t>(dim);
    const hipError_t e = rr::launch_norm_join(j, k, s);
    if (e != hipSuccess) return hip_fail(e, "layer_norm_grad: weight");
  }
  return ok();
}

// ---------------------------------------------------------------------------
// Gated projections.

constexpr uint64_t kMaxTokens = 1ull << 23;
constexpr uint64_t kMaxWidth = 1ull << 20;   // dim
constexpr uint64_t kMaxFeatures = 1ull << 19;  // 256 rows of both products' gradients span less than 2^31 bytes
constexpr uint64_t kMaxMatrix = 1ull << 36;

rr_status_t check_gated_shape(int p, size_t tokens, size_t dim, size_t ffn, rr_act_t act, rr_dtype_t dtype) {
  rr_status_t st;
  if ((st = check_p(p)) || (st = check_float_dtype(dtype, "the gated projections"))) return st;
  if (act != RR_SILU && act != RR_GELU)
    return fail(RR_ERROR_UNSUPPORTED, "unknown activation %d", static_cast<int>(act));
  if (dim < 1 || dim > kMaxWidth) return fail(RR_ERROR_INVALID_ARGUMENT, "dim=%zu outside [1, 2^20]", dim);
  if (ffn < 1 || ffn > kMaxFeatures) return fail(RR_ERROR_INVALID_ARGUMENT, "ffn=%zu outside [1, 2^19]", ffn);
  if (tokens > kMaxTokens) return fail(RR_ERROR_INVALID_ARGUMENT, "tokens=%zu exceeds 2^23", tokens);
  if (static_cast<uint64_t>(tokens) * dim > kMaxMatrix || static_cast<uint64_t>(ffn) * dim > kMaxMatrix ||
      static_cast<uint64_t>(tokens) * ffn > kMaxMatrix)
    return fail(RR_ERROR_INVALID_ARGUMENT, "tokens*dim, ffn*dim or tokens*ffn exceeds 2^36");
  return RR_SUCCESS;
}

// The shards' buffers, `per` elements a feature; ranks without features may be NULL.
rr_status_t check_shards(const void* const* bufs, const char* what, const rr::GatedShards& sh, uint64_t per, size_t esz,
                         int id, std::vector<Range>& ranges) {
  if (!bufs) return fail(RR_ERROR_INVALID_ARGUMENT, "%s is NULL", what);
  for (int r = 0; r < sh.p; ++r) {
    if (sh.rows[r] == 0 || per == 0) continue;
    const rr_status_t st = check_buf(bufs[r], esz, what, r);
    if (st) return st;
    ranges.push_back(range_of(bufs[r], sh.rows[r] * per * esz, id));
  }
  return RR_SUCCESS;
}

// The kept products: both or none, in the storage type or float32.
rr_status_t check_pre(const void* pre_gates, const void* pre_ups, rr_dtype_t pre_dtype, rr_dtype_t dtype) {
  if (!pre_gates != !pre_ups) return fail(RR_ERROR_INVALID_ARGUMENT, "pre_gates and pre_ups: one of them is NULL");
  if (pre_gates && pre_dtype != dtype && pre_dtype != RR_FLOAT32)
    return fail(RR_ERROR_UNSUPPORTED, "pre_dtype %d is neither the dtype nor float32", static_cast<int>(pre_dtype));
  return RR_SUCCESS;
}

bool never(const Range&, const Range&) { return false; }

struct GatedCall {
  rr::GatedPlan pl;
  rr::GatedShards sh;  // the caller's weights
  const void* hidden;
  bool pack;
  bool rows_too;  // the next copy of weights copies the hidden rows with it, into pack_x
  Kind k;
  rr::GatedAct act;
  char* ws;
  hipStream_t s;
};

// What both directions read, and the workspace.
rr_status_t gated_inputs(GatedCall& c, const void* hidden, const void* const* gates, const void* const* ups,
                         rr_act_t act, int p, size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, bool grad,
                         bool kept, void* workspace, size_t workspace_bytes, rr_stream_t stream,
                         std::vector<Range>& ins) {
  rr_status_t st;
  if ((st = check_gated_shape(p, tokens, dim, ffn, act, dtype))) return st;
  const size_t esz = rr::elem_size(dtype);
  const auto plan = [&](bool pack) {
    rr::plan_gated(c.pl, p, static_cast<uint32_t>(tokens), static_cast<uint32_t>(dim), static_cast<uint32_t>(ffn),
                   dtype, grad, pack, kept);
  };
  plan(false);
  if ((st = check_shards(gates, "gate_weights", c.pl.sh, dim, esz, -1, ins)) ||
      (st = check_shards(ups, "up_weights", c.pl.sh, dim, esz, -2, ins)))
    return st;
  c.pack = (dim * esz) % 16 != 0;
  if (tokens > 0) {
    if ((st = check_one(hidden, "hidden", esz, tokens * dim * esz, -3, ins))) return st;
    c.pack = c.pack || !aligned16(hidden);
  }
  for (int r = 0; r < p; ++r)
    if (c.pl.sh.rows[r]) c.pack = c.pack || !aligned16(gates[r]) || !aligned16(ups[r]);
  if ((st = check_workspace(workspace, workspace_bytes,
                            rr_gated_linear_workspace_size(p, tokens, dim, ffn, dtype, !grad ? 0 : kept ? 2 : 1))))
    return st;
  if (c.pack) plan(true);
  c.sh = c.pl.sh;
  for (int r = 0; r < p; ++r) {
    c.sh.gate[r] = gates[r];
    c.sh.up[r] = ups[r];
  }
  c.hidden = hidden;
  c.rows_too = false;
  c.k = kind_of(dtype);
  c.act = act == RR_SILU ? rr::GatedAct::kSilu : rr::GatedAct::kGelu;
  c.ws = static_cast<char*>(workspace);
  c.s = reinterpret_cast<hipStream_t>(stream);
  return RR_SUCCESS;
}

// The weights of the padded features [f0, f1) in aligned rows: the pointers then
// are where row 0 of a shard would lie (only rows of the piece are read).
hipError_t gated_piece(GatedCall& c, uint32_t f0, uint32_t f1, bool copy, rr::GatedShards& out) {
  out = c.sh;
  if (!c.pack) return hipSuccess;
  const uint64_t row = static_cast<uint64_t>(c.pl.dim_pad) * c.pl.esz;
  hipError_t e = hipSuccess;
  if (copy) {
    rr::GatedPackArgs a;
    a.sh = c.sh;
    a.out = c.ws + c.pl.pack_w;
    a.out_stride = row;
    a.dim = c.pl.dim;
    a.f0 = f0;
    a.f1 = f1;
    a.x = c.hidden;
    a.x_out = c.ws + c.pl.pack_x;
    a.tokens = c.rows_too ? c.pl.tokens : 0;
    c.rows_too = false;
    e = rr::launch_gated_pack(a, c.k, c.s);
  }
  const uintptr_t base = reinterpret_cast<uintptr_t>(c.ws + c.pl.pack_w);
  for (int r = 0; r < c.sh.p; ++r) {
    const uint64_t first = static_cast<uint64_t>(c.sh.off[r]) * row - static_cast<uint64_t>(f0) * row;
    out.gate[r] = reinterpret_cast<const void*>(base + first);
    out.up[r] = reinterpret_cast<const void*>(base + (f1 - f0) * row + first);
  }
  return e;
}

// The forward kernels' outputs, as `a` says where.
hipError_t gated_forward(GatedCall& c, rr::GatedArgs& a, rr::GatedMode m) {
  const rr::GatedPlan& pl = c.pl;
  const uint32_t all = pl.sh.off[pl.sh.p];
  a.sh = c.sh;
  a.x = c.hidden;
  a.x_stride = a.w_stride = static_cast<uint64_t>(pl.dim) * pl.esz;
  a.dim = pl.dim;
  a.tokens = pl.tokens;
  a.kbytes = static_cast<uint32_t>(a.x_stride);
  if (pl.forward_tile == rr::GatedTile::kFew) {
    a.f0 = 0;
    a.f1 = all;
    return rr::launch_gated(a, c.k, c.act, m, pl.forward_tile, c.s);
  }
  if (c.pack) {
    a.x = c.ws + pl.pack_x;
    a.x_stride = a.w_stride = static_cast<uint64_t>(pl.dim_pad) * pl.esz;
    a.kbytes = static_cast<uint32_t>(a.x_stride);
  }
  for (uint32_t f0 = 0; f0 < all; f0 += pl.piece) {
    const uint32_t f1 = std::min(all, f0 + pl.piece);
    hipError_t e = gated_piece(c, f0, f1, true, a.sh);
    if (e != hipSuccess) return e;
    // large tiles and, for a last round that would leave most of the chip idle, small ones
    const bool f32 = c.k == Kind::kF32;
    const uint32_t fm = rr::gated_tail(2 * f0, 2 * f1, pl.tokens, tiles_over(pl.dim, 64), pl.forward_tile, f32,
                                       a.has_pre ? rr::GatedUse::kForwardWide : rr::GatedUse::kForward) / 2;
    for (int tail = 0; tail < 2; ++tail) {
      const rr::GatedTile t = tail ? rr::gated_small(f32) : pl.forward_tile;
      a.f0 = tail ? fm : f0;
      a.f1 = tail ? f1 : fm;
      if (a.f0 == a.f1) continue;
      a.tiles_m = tiles_over(2ull * (a.f1 - a.f0), rr::tile_m(t));
      a.tiles_n = tiles_over(pl.tokens, rr::tile_n(t));
      if ((e = rr::launch_gated(a, c.k, c.act, m, t, c.s)) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

// The hidden rows as they are, into aligned rows.
rr::GatedRowsArgs gated_rows(const GatedCall& c, void* out) {
  rr::GatedRowsArgs a;
  memset(&a, 0, sizeof(a));
  a.x = c.hidden;
  a.out = out;
  a.out_stride = static_cast<uint64_t>(c.pl.dim_pad) * c.pl.esz;
  a.tokens = c.pl.tokens;
  a.dim = c.pl.dim;
  return a;
}

rr_status_t gated_body(const void* hidden, const void* const* gates, const void* const* ups, void* const* recvbufs,
                       void* const* pre_gates, void* const* pre_ups, rr_dtype_t pre_dtype, rr_act_t act, int p,
                       size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, void* workspace,
                       size_t workspace_bytes, rr_stream_t stream) {
  rr_status_t st;
  GatedCall c;
  std::vector<Range> ins, outs;
  if ((st = gated_inputs(c, hidden, gates, ups, act, p, tokens, dim, ffn, dtype, false, pre_gates != nullptr,
                         workspace, workspace_bytes, stream, ins)))
    return st;
  if ((st = check_pre(pre_gates, pre_ups, pre_dtype, dtype))) return st;
  const size_t esz = rr::elem_size(dtype), pre_esz = rr::elem_size(pre_dtype);
  if ((st = check_shards(recvbufs, "recvbufs", c.sh, tokens, esz, -4, outs))) return st;
  if (pre_gates && ((st = check_shards(pre_gates, "pre_gates", c.sh, tokens, pre_esz, -5, outs)) ||
                    (st = check_shards(pre_ups, "pre_ups", c.sh, tokens, pre_esz, -6, outs))))
    return st;
  if (tokens == 0) return ok();
  if (workspace && workspace_bytes) outs.push_back(range_of(workspace, workspace_bytes, -7));
  if ((st = check_aliasing_sorted(outs, ins, never))) return st;
  if (log_launches())
    fprintf(stderr, "[rr] gated_linear: p=%d tokens=%zu dim=%zu ffn=%zu tile=%d copy=%d\n", p, tokens, dim, ffn,
            static_cast<int>(c.pl.forward_tile), c.pack ? 1 : 0);
  rr::GatedArgs a;
  memset(&a, 0, sizeof(a));
  for (int r = 0; r < p; ++r) {
    a.h[r] = recvbufs[r];
    a.a[r] = pre_gates ? pre_gates[r] : nullptr;
    a.u[r] = pre_ups ? pre_ups[r] : nullptr;
  }
  a.has_h = 1;
  a.has_pre = pre_gates ? 1 : 0;
  a.pre32 = pre_dtype == RR_FLOAT32 ? 1 : 0;
  c.rows_too = c.pack && c.pl.forward_tile != rr::GatedTile::kFew;
  const hipError_t e = gated_forward(c, a, rr::GatedMode::kForward);
  if (e != hipSuccess) return hip_fail(e, "gated_linear");
  return ok();
}

rr_status_t gated_grad_body(const void* hidden, const void* const* gates, const void* const* ups,
                            const void* const* grad_outs, const void* const* pre_gates, const void* const* pre_ups,
                            rr_dtype_t pre_dtype, void* dhidden, void* const* dgates, void* const* dups, rr_act_t act,
                            int p, size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            rr_stream_t stream) {
  rr_status_t st;
  GatedCall c;
  std::vector<Range> ins, outs;
  if ((st = gated_inputs(c, hidden, gates, ups, act, p, tokens, dim, ffn, dtype, true,
                         pre_gates != nullptr, workspace, workspace_bytes, stream, ins)))
    return st;
  if ((st = check_pre(pre_gates, pre_ups, pre_dtype, dtype))) return st;
  if (!dgates != !dups)
    return fail(RR_ERROR_INVALID_ARGUMENT, "dgate_weights and dup_weights: one of them is NULL");
  if (!dhidden && !dgates) return fail(RR_ERROR_INVALID_ARGUMENT, "dhidden and the weights' gradients are all NULL");
  const size_t esz = rr::elem_size(dtype), pre_esz = rr::elem_size(pre_dtype);
  const bool pre32 = pre_dtype == RR_FLOAT32;
  if ((st = check_shards(grad_outs, "grad_outs", c.sh, tokens, esz, -4, ins))) return st;
  if (pre_gates && ((st = check_shards(pre_gates, "pre_gates", c.sh, tokens, pre_esz, -5, ins)) ||
                    (st = check_shards(pre_ups, "pre_ups", c.sh, tokens, pre_esz, -6, ins))))
    return st;
  if (dhidden && tokens > 0 && (st = check_one(dhidden, "dhidden", esz, tokens * dim * esz, -7, outs))) return st;
  if (dgates && ((st = check_shards(dgates, "dgate_weights", c.sh, dim, esz, -8, outs)) ||
                 (st = check_shards(dups, "dup_weights", c.sh, dim, esz, -9, outs))))
    return st;
  if (workspace && workspace_bytes) outs.push_back(range_of(workspace, workspace_bytes, -10));
  if ((st = check_aliasing_sorted(outs, ins, never))) return st;
  if (tokens == 0 && !dgates) return ok();

  const rr::GatedPlan& pl = c.pl;
  const bool f16 = dtype == RR_FLOAT16, f32 = dtype == RR_FLOAT32;
  const uint64_t row = static_cast<uint64_t>(pl.dim_pad) * esz;
  const uint32_t all = pl.sh.off[p];
  if (log_launches())
    fprintf(stderr, "[rr] gated_linear_grad: p=%d tokens=%zu dim=%zu ffn=%zu tiles=%d/%d/%d splits=%u kept=%d copy=%d\n",
            p, tokens, dim, ffn, static_cast<int>(pl.forward_tile), static_cast<int>(pl.hidden_tile),
            static_cast<int>(pl.weight_tile), pl.splits, pre_gates ? 1 : 0, c.pack ? 1 : 0);
  char* const grad = c.ws + pl.grad;
  float* const row_max = f16 ? reinterpret_cast<float*>(c.ws + pl.row_max) : nullptr;
  int32_t* const row_exp = f16 && dgates ? reinterpret_cast<int32_t*>(c.ws + pl.row_exp) : nullptr;
  int32_t* const scale = f16 ? reinterpret_cast<int32_t*>(c.ws + pl.scale) : nullptr;
  hipError_t e = hipSuccess;
  bool packed = false;  // the weights' only piece lies in the workspace
  // the forward kernels read aligned rows
  const bool copied = tokens > 0 && c.pack && !pre_gates && pl.forward_tile != rr::GatedTile::kFew;
  if (tokens > 0) {
    c.rows_too = copied;
    if (!pre_gates) {
      // the products again; their gradients at once, but float16's, which wait for their row's scale
      rr::GatedArgs a;
      memset(&a, 0, sizeof(a));
      for (int r = 0; r < p; ++r) a.h[r] = const_cast<void*>(grad_outs[r]);
      a.pre = f16 ? c.ws + pl.pre : grad;
      a.pre_ld = pl.ld;
      a.has_pre = 1;
      a.pre32 = f16 || f32 ? 1 : 0;
      if ((e = gated_forward(c, a, f16 ? rr::GatedMode::kForward : rr::GatedMode::kGrad)) != hipSuccess)
        return hip_fail(e, "gated_linear_grad: forward");
      packed = pl.piece >= all && pl.forward_tile != rr::GatedTile::kFew;
    }
  }
  if (tokens > 0 && (pre_gates || f16)) {
    rr::GatedGradArgs g;
    memset(&g, 0, sizeof(g));
    for (int r = 0; r < p; ++r) {
      g.dh[r] = grad_outs[r];
      g.a[r] = pre_gates ? pre_gates[r] : nullptr;
      g.u[r] = pre_ups ? pre_ups[r] : nullptr;
    }
    memcpy(g.off, pl.sh.off, sizeof(g.off));
    memcpy(g.rows, pl.sh.rows, sizeof(g.rows));
    g.p = p;
    g.pre = pre_gates ? nullptr : reinterpret_cast<const float*>(c.ws + pl.pre);
    g.pre32 = pre32 ? 1 : 0;
    g.grad = grad;
    g.ld = pl.ld;
    g.tokens = pl.tokens;
    g.row_max = row_max;
    g.row_exp = row_exp;
    g.x = hidden;
    g.dim = pl.dim;
    if ((e = rr::launch_gated_grad(g, c.k, c.act, c.s)) != hipSuccess) return hip_fail(e, "gated_linear_grad: activation");
  }
  // The rows that the weights' gradients read: the hidden states themselves, or a
  // copy, in aligned rows or scaled.
  const bool copy = dgates && tokens > 0 && (f16 || (c.pack && !copied));
  rr::GatedRowsArgs rows = gated_rows(c, c.ws + (f16 ? pl.xs : pl.pack_x));
  rows.row_max = row_max;
  rows.row_exp = row_exp;
  rows.scale = scale;
  const bool brief = tokens > 0 && tokens <= rr::kGatedRideTokens;
  const bool ride_copy = copy && brief && dhidden && pl.hidden_tile != rr::GatedTile::k256x256;
  if (f16 && dgates && !ride_copy && (e = rr::launch_gated_scale(row_exp, pl.tokens, scale, c.s)) != hipSuccess)
    return hip_fail(e, "gated_linear_grad: scale");
  c.rows_too = copy && !ride_copy && !f16 && dhidden;  // (dhidden's weights are copied then)
  if (copy && !ride_copy && !c.rows_too && (e = rr::launch_gated_rows(rows, c.k, c.s)) != hipSuccess)
    return hip_fail(e, "gated_linear_grad: copy");
  rr::GatedJoinArgs j;
  memset(&j, 0, sizeof(j));
  bool ride_join = false;
  if (dhidden && tokens > 0) {
    const bool direct = pl.direct();
    ride_join = !direct && dgates && pl.weight_tile != rr::GatedTile::k256x256 &&
                tokens <= (f16 ? rr::kGatedRideTokens : rr::kGatedJoinTokens);
    rr::GatedHiddenArgs h;
    memset(&h, 0, sizeof(h));
    h.ld = pl.ld;
    h.w_stride = c.pack ? row : dim * esz;
    h.acc = reinterpret_cast<float*>(c.ws + pl.acc);
    h.split_stride = static_cast<uint64_t>(tokens) * pl.acc_ld;
    h.acc_ld = pl.acc_ld;
    h.out = direct ? dhidden : nullptr;
    h.row_max = row_max;
    h.tokens = pl.tokens;
    h.dim = pl.dim;
    h.tiles_m = tiles_over(dim, rr::tile_m(pl.hidden_tile));
    h.tiles_n = tiles_over(tokens, rr::tile_n(pl.hidden_tile));
    h.splits = pl.splits;
    if (ride_copy) {
      // a multiple of the XCDs, so that the tiles keep their places
      h.riders = (tiles_over(tokens, rr::kGatedRiderRows) + 7) / 8 * 8;
      h.copy = rows;
    }
    for (uint32_t f0 = 0; f0 < all; f0 += pl.piece) {
      const uint32_t f1 = std::min(all, f0 + pl.piece);
      if ((e = gated_piece(c, f0, f1, !packed, h.sh)) != hipSuccess) return hip_fail(e, "gated_linear_grad: copy");
      h.c0 = 2 * f0;
      h.c1 = 2 * f1;
      h.grad = grad + static_cast<uint64_t>(h.c0) * esz;
      h.add = f0 > 0 ? 1 : 0;
      if ((e = rr::launch_gated_hidden(h, c.k, pl.hidden_tile, c.s)) != hipSuccess)
        return hip_fail(e, "gated_linear_grad: dhidden");
      h.riders = 0;
    }
    if (!direct) {
      j.acc = h.acc;
      j.split_stride = h.split_stride;
      j.acc_ld = pl.acc_ld;
      j.row_max = row_max;
      j.out = dhidden;
      j.tokens = pl.tokens;
      j.dim = pl.dim;
      j.splits = pl.splits;
      if (!ride_join && (e = rr::launch_gated_join(j, c.k, c.s)) != hipSuccess)
        return hip_fail(e, "gated_linear_grad: dhidden");
    }
  }
  if (dgates) {
    rr::GatedWeightArgs w;
    memset(&w, 0, sizeof(w));
    w.x = copy ? rows.out : copied ? c.ws + pl.pack_x : hidden;
    w.x_stride = copy || copied ? row : dim * esz;
    for (int r = 0; r < p; ++r) {
      w.dgate[r] = dgates[r];
      w.dup[r] = dups[r];
    }
    memcpy(w.off, pl.sh.off, sizeof(w.off));
    memcpy(w.rows, pl.sh.rows, sizeof(w.rows));
    w.p = p;
    w.grad = grad;
    w.ld = pl.ld;
    w.scale = scale;
    w.acc = reinterpret_cast<float*>(c.ws + pl.weight_acc);
    w.acc_stride = pl.ld * pl.acc_ld;
    w.acc_ld = pl.acc_ld;
    w.tokens = pl.tokens;
    w.dim = pl.dim;
    const uint32_t c1 = 2 * all;
    const uint32_t cm = rr::gated_tail(0, c1, pl.dim, tiles_over(pl.tokens, 64), pl.weight_tile, f32,
                                       rr::GatedUse::kWeights);
    if (ride_join) {
      // (one launch: its tiles are small)
      const bool many = j.splits >= rr::kGatedJoinMany;
      w.join = j;
      w.join_cols = tiles_over(dim, many ? 256 : 1024);
      w.riders = static_cast<uint32_t>((tokens * w.join_cols + 7) / 8 * 8);  // a multiple of the XCDs
      // Behind the tiles where those leave places for workgroups free, two a compute
      // unit, else in front of them.
      const uint32_t tiles = tiles_over(dim, rr::tile_m(pl.weight_tile)) * tiles_over(c1, rr::tile_n(pl.weight_tile)) *
                             pl.weight_splits;
      w.rider0 = tiles < 2 * 256 ? tiles : 0;
    }
    for (int tail = 0; tail < 2; ++tail) {
      const rr::GatedTile t = tail ? rr::gated_small(f32) : pl.weight_tile;
      w.c0 = tail ? cm : 0;
      w.c1 = tail ? c1 : cm;
      if (w.c0 == w.c1) continue;
      w.tiles_m = tiles_over(dim, rr::tile_m(t));
      w.tiles_n = tiles_over(w.c1 - w.c0, rr::tile_n(t));
      w.splits = pl.weight_splits;
      if ((e = rr::launch_gated_weight(w, c.k, t, c.s)) != hipSuccess) return hip_fail(e, "gated_linear_grad: weights");
      if (w.splits > 1 && (e = rr::launch_gated_weight_join(w, c.k, c.s)) != hipSuccess)
        return hip_fail(e, "gated_linear_grad: weights");
    }
  }
  return ok();
}

}  // namespace

extern "C" {

rr_status_t rr_layer_norm(const void* const* sendbufs, const void* weight, const void* bias, void* const* recvbufs,
                          float* mean, float* rstd, int p, size_t rows, size_t dim, double eps, int center,
                          rr_dtype_t dtype, rr_stream_t stream) {
  return guarded([&] {
    return norm_body(sendbufs, weight, bias, recvbufs, mean, rstd, p, rows, dim, eps, center, dtype, stream);
  });
}

rr_status_t rr_layer_norm_grad(const void* const* grad_outs, const void* const* sendbufs, const void* weight,
                               const float* mean, const float* rstd, const void* const* residuals,
                               void* const* grad_ins, void* dweight, void* dbias, int p, size_t rows, size_t dim,
                               int center, rr_dtype_t dtype, void* workspace, size_t workspace_bytes,
                               rr_stream_t stream) {
  return guarded([&] {
    return norm_grad_body(grad_outs, sendbufs, weight, mean, rstd, residuals, grad_ins, dweight, dbias, p, rows, dim,
                          center, dtype, workspace, workspace_bytes, stream);
  });
}

size_t rr_layer_norm_grad_workspace_size(int p, size_t rows, size_t dim, rr_dtype_t dtype) {
  if (check_norm_shape(p, rows, dim, dtype)) return 0;
  ok();
  const uint32_t grid =
      rr::norm_grad_grid(static_cast<uint32_t>(rows * static_cast<size_t>(p)), static_cast<uint32_t>(dim), kind_of(dtype));
  return static_cast<size_t>(grid) * rr::norm_line(static_cast<uint32_t>(dim)) * sizeof(float);
}

rr_status_t rr_gated_linear(const void* hidden, const void* const* gate_weights, const void* const* up_weights,
                            void* const* recvbufs, void* const* pre_gates, void* const* pre_ups, rr_dtype_t pre_dtype,
                            rr_act_t act, int p, size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, void* workspace,
                            size_t workspace_bytes, rr_stream_t stream) {
  return guarded([&] {
    return gated_body(hidden, gate_weights, up_weights, recvbufs, pre_gates, pre_ups, pre_dtype, act, p, tokens, dim,
                      ffn, dtype, workspace, workspace_bytes, stream);
  });
}

rr_status_t rr_gated_linear_grad(const void* hidden, const void* const* gate_weights, const void* const* up_weights,
                                 const void* const* grad_outs, const void* const* pre_gates,
                                 const void* const* pre_ups, rr_dtype_t pre_dtype, void* dhidden,
                                 void* const* dgate_weights, void* const* dup_weights, rr_act_t act, int p,
                                 size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, void* workspace,
                                 size_t workspace_bytes, rr_stream_t stream) {
  return guarded([&] {
    return gated_grad_body(hidden, gate_weights, up_weights, grad_outs, pre_gates, pre_ups, pre_dtype, dhidden,
                           dgate_weights, dup_weights, act, p, tokens, dim, ffn, dtype, workspace, workspace_bytes, stream);
  });
}

size_t rr_gated_linear_workspace_size(int p, size_t tokens, size_t dim, size_t ffn, rr_dtype_t dtype, int grad) {
  if (check_gated_shape(p, tokens, dim, ffn, RR_SILU, dtype)) return 0;
  ok();
  rr::GatedPlan aligned, packed;
  const auto plan = [&](rr::GatedPlan& pl, bool pack) {
    rr::plan_gated(pl, p, static_cast<uint32_t>(tokens), static_cast<uint32_t>(dim), static_cast<uint32_t>(ffn), dtype,
                   grad != 0, pack, grad == 2);
  };
  plan(packed, true);
  plan(aligned, false);
  return std::max(aligned.total, packed.total);
}

}  // extern "C"
