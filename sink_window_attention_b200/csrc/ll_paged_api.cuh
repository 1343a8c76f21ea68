// ll_paged_api.cuh — host side of the token-stream entry points (the last part
// of ll_api.cu: uses its error, alignment and per-device helpers).
#pragma once

#include "ll_paged_attention.cuh"
#include "ll_paged_prefill.cuh"
#include "ll_tokens.cuh"

namespace {

static_assert(LL_MAX_TOKEN_HEADS == ll::kMaxTokenHeads && LL_MAX_TOKEN_PAIRS == ll::kMaxTokenPairs, "header limits");

ll_status make_token_rope(const ll_token_rope_desc* r, int D, int transpose, ll::TokenRope* out) {
  std::memset(out, 0, sizeof(*out));
  if (r == nullptr) return LL_OK;  // no rotation
  if (r->rot_dim < 16 || r->rot_dim % 16 != 0 || r->rot_dim > 2 * LL_MAX_TOKEN_PAIRS || r->rot_dim > D)
    return fail(LL_ERR_INVALID_ARG, "rot_dim = %d must be a multiple of 16 in [16, min(%d, D = %d)]", r->rot_dim,
                2 * LL_MAX_TOKEN_PAIRS, D);
  if (r->layout != LL_ROPE_INTERLEAVED && r->layout != LL_ROPE_HALF)
    return fail(LL_ERR_INVALID_ARG, "unknown rope layout %d", r->layout);
  if (!std::isfinite(r->amplitude)) return fail(LL_ERR_INVALID_ARG, "rope amplitude must be finite");
  out->rot = r->rot_dim;
  out->half = r->layout == LL_ROPE_HALF;
  out->amp = r->amplitude;
  out->sign = transpose ? -1.f : 1.f;
  for (int i = 0; i < r->rot_dim / 2; ++i) out->turns[i] = r->turns[i];
  return LL_OK;
}

ll_status check_paged_cache(const ll_paged_cache* c) {
  if (c == nullptr) return fail(LL_ERR_INVALID_ARG, "cache is NULL");
  if (c->k == nullptr || c->v == nullptr) return fail(LL_ERR_INVALID_ARG, "cache k/v pointer is NULL");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(LL_ERR_INVALID_ARG, "cache k/v must be 16-byte aligned");
  if (c->dtype != LL_BF16 && c->dtype != LL_FP8_E4M3)
    return fail(LL_ERR_INVALID_ARG, "a paged cache is BF16 or FP8_E4M3 (got dtype %d)", (int)c->dtype);
  if (c->dtype == LL_FP8_E4M3 && (c->k_scale == nullptr || c->v_scale == nullptr))
    return fail(LL_ERR_INVALID_ARG, "an FP8 cache needs k_scale and v_scale");
  if (c->dtype == LL_FP8_E4M3 && (!aligned4(c->k_scale) || !aligned4(c->v_scale)))
    return fail(LL_ERR_INVALID_ARG, "k_scale and v_scale must be 4-byte aligned");
  if (c->n_pages < 1 || c->H < 1) return fail(LL_ERR_INVALID_ARG, "cache sizes must be positive (n_pages=%d H=%d)",
                                              c->n_pages, c->H);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(LL_ERR_INVALID_ARG, "page_size = %d must be 16, 32, 64 or 128", c->page_size);
  if (c->D != 64 && c->D != 128) return fail(LL_ERR_INVALID_ARG, "D = %d must be 64 or 128", c->D);
  if (c->H > LL_MAX_TOKEN_HEADS) return fail(LL_ERR_INVALID_ARG, "H = %d exceeds %d", c->H, LL_MAX_TOKEN_HEADS);
  if (static_cast<long long>(c->n_pages) * c->H * (c->page_size / 16) > INT_MAX)
    return fail(LL_ERR_INVALID_ARG, "n_pages x H x page_size / 16 = %lld exceeds 2^31 - 1",
                static_cast<long long>(c->n_pages) * c->H * (c->page_size / 16));
  return LL_OK;
}

ll_status check_batch(const ll_token_batch* t) {
  if (t == nullptr) return fail(LL_ERR_INVALID_ARG, "batch is NULL");
  if (t->q_start == nullptr || t->kv_len == nullptr || t->page_table == nullptr)
    return fail(LL_ERR_INVALID_ARG, "q_start, kv_len and page_table must be non-NULL");
  if (!aligned4(t->q_start) || !aligned4(t->kv_len) || !aligned4(t->page_table))
    return fail(LL_ERR_INVALID_ARG, "q_start, kv_len and page_table must be 4-byte aligned");
  if (t->B < 1 || t->max_pages < 1) return fail(LL_ERR_INVALID_ARG, "B = %d and max_pages = %d must be positive", t->B,
                                                t->max_pages);
  if (t->B > 65535) return fail(LL_ERR_INVALID_ARG, "B = %d exceeds 65535", t->B);
  if (t->total_q < 0 || t->max_q < 0 || t->max_kv < 0)
    return fail(LL_ERR_INVALID_ARG, "total_q, max_q and max_kv must be >= 0");
  return LL_OK;
}

ll_status check_rows(const char* what, const void* x, long long stride, int H, int D) {
  if (x == nullptr) return fail(LL_ERR_INVALID_ARG, "%s must be non-NULL", what);
  if (!aligned16(x)) return fail(LL_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  if (stride % 8 != 0 || stride < static_cast<long long>(H) * D)
    return fail(LL_ERR_INVALID_ARG, "the row stride %lld of %s must be a multiple of 8 and at least H * D = %lld", stride,
                what, static_cast<long long>(H) * D);
  return LL_OK;
}

// Keys of a sequence that may exist: the kernels round up to whole tiles in 32 bits.
int max_key(const ll_token_batch* t, int page_size) {
  const long long cap = static_cast<long long>(t->max_pages) * page_size;
  const long long n = t->max_kv < cap ? t->max_kv : cap;
  return static_cast<int>(n < INT_MAX - 256 ? n : INT_MAX - 256);
}

ll::TokenBatch to_batch(const ll_token_batch* t, int page_size) {
  ll::TokenBatch b;
  b.q_start = t->q_start;
  b.kv_len = t->kv_len;
  b.page_table = t->page_table;
  b.B = t->B;
  b.max_pages = t->max_pages;
  b.total_q = t->total_q;
  b.max_q = t->max_q < t->total_q ? t->max_q : t->total_q;
  b.max_key = max_key(t, page_size);
  return b;
}

ll::PagedPool to_pool(const ll_paged_cache* c) {
  ll::PagedPool p;
  p.k = c->k;
  p.v = c->v;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  p.H = c->H;
  p.D = c->D;
  return p;
}

// Dynamic shared memory above the 48 KiB that a launch may use unasked.
template <class K>
ll_status allow_smem(K kern, int bytes, std::atomic<unsigned long long>& done) {
  return once_per_device(done, [&]() -> ll_status {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return check_launch("cudaFuncSetAttribute");
    return LL_OK;
  });
}

// How a call's rows and keys are divided among blocks. A function of the host's
// bounds alone, so the workspace size is known before the call.
// Rows of a sequence and K/V head up to which the decode kernel is taken. 8 sequences of
// 2000 to 8000 keys, 8 K/V heads of 128, decode (tiles of 128 rows): 8-bit 48 rows 68 us
// (80), 64 rows 82 (82), 96 rows 120 (84); bf16 32 rows 60 (70), 48 rows 80 (70), 64 rows
// 100 (72); heads of 64, bf16 48 rows 51 (64), 64 rows 62 (65). From 33 to 48 rows over a
// bf16 pool of heads of 128 the tiles would be faster, but they keep a rotated q in one term.
constexpr int kDecodeRows = 48;
// Over short ranges, which stay in L2, it is taken for more rows where its waves of
// blocks (6 us to start and end one, 0.08 us per 16 keys of 128 elements) take less than
// the tile kernel's (10 us, 2.4 us per 128 keys). 1000 keys, bf16, decode (tiles): one
// sequence, 8 K/V heads of 128, 256 rows 19 us (21), 512 rows 23 (27), 1024 rows 41 (35); six
// of 512 rows 115 (29), 12 heads of 64 79 (25). The estimate leaves out what blocks that read the
// same keys cost L2, and what a split costs the tile kernel: with six full sequences of 256
// rows it takes decode, 62 us (45), heads of 64 49 (49).
constexpr long long kShortRange = 1024;

// Blocks of the decode kernel that an SM holds.
int decode_blocks(const ll_paged_cache* c, int rows) {
  const bool e4m3 = c->dtype == LL_FP8_E4M3;
  if (c->D == 128)
    return e4m3 ? (rows == 8 ? ll::DecodeTraits<128, true, 8>::BLOCKS : ll::DecodeTraits<128, true, 16>::BLOCKS)
                : (rows == 8 ? ll::DecodeTraits<128, false, 8>::BLOCKS : ll::DecodeTraits<128, false, 16>::BLOCKS);
  return e4m3 ? (rows == 8 ? ll::DecodeTraits<64, true, 8>::BLOCKS : ll::DecodeTraits<64, true, 16>::BLOCKS)
              : (rows == 8 ? ll::DecodeTraits<64, false, 8>::BLOCKS : ll::DecodeTraits<64, false, 16>::BLOCKS);
}

struct AttnPlan {
  bool tiles;      // 128-row tensor-memory tiles; else warp tiles of 8 or 16 rows
  bool clustered;  // the pieces of a unit are joined by a cluster on chip; else through the workspace
  int row_tile, key_tile, row_tiles, chunk, chunk0, nsplit;
};

// The plan for key ranges of at most `span` keys (0: no such bound).
AttnPlan plan_for_span(const ll_paged_cache* c, const ll_token_batch* t, int Hq, long long span) {
  AttnPlan a;
  const int group = Hq / c->H;
  const long long max_q = t->max_q < t->total_q ? t->max_q : t->total_q;
  const long long rows = max_q * group, keys = max_key(t, c->page_size);
  // tiles in a range at most: a span's two ends and the sinks' end may each cut one
  auto tiles_of = [&](long long tile) {
    const long long n = span > 0 && span + 3 * tile < keys ? span + 3 * tile : keys;
    return n > 0 ? (n + tile - 1) / tile : 1;
  };
  auto waves_of = [&](long long row_tile, long long slots) {
    return ((rows + row_tile - 1) / row_tile * t->B * c->H + slots - 1) / slots;
  };
  a.tiles = rows > kDecodeRows;
  if (a.tiles && 16 * tiles_of(16) <= kShortRange)
    a.tiles = waves_of(256, num_sms()) * (1000 + 240 * tiles_of(128)) <
              waves_of(16, 3ll * num_sms()) * (600 + 8 * tiles_of(16) * c->D / 128);
  a.row_tile = a.tiles ? 256 : (rows <= 8 ? 8 : 16);
  a.key_tile = a.tiles ? 128 : 16;
  a.row_tiles = static_cast<int>((rows + a.row_tile - 1) / a.row_tile);
  const long long nt = tiles_of(a.key_tile);
  const long long units = static_cast<long long>(t->B) * c->H * (a.row_tiles > 0 ? a.row_tiles : 1);
  long long chunk = nt, chunk0 = 0;  // chunk0 0: like the others
  if (!a.tiles) {
    // Long ranges: three waves of blocks, whole ones so that equal lengths leave no block
    // over, several so that ragged ones even out (one sequence is as long as itself: one
    // wave). Where that leaves less than 512 keys to a piece the join would cost more than
    // it saves, and latency counts: no more blocks than run at once, at least 128 keys
    // each (two tiles per warp), in a cluster (8 blocks are portable) where they fit one.
    const long long slots = decode_blocks(c, a.row_tile) * static_cast<long long>(num_sms());
    const long long many = (t->B > 1 ? 3 : 1) * slots / units, few = slots / units;
    if (many > 1 && nt >= 32 * many) {
      chunk = (nt + many - 1) / many;
    } else {
      long long pieces = nt / 8 < few ? nt / 8 : few;
      if (pieces > 8 && (pieces <= 12 || nt <= 8 * 16)) pieces = 8;
      if (pieces > 8 && nt < 24 * pieces) pieces = nt / 24 > 8 ? nt / 24 : 8;
      chunk = pieces > 1 ? (nt + pieces - 1) / pieces : nt;
    }
  } else {
    // one block per SM: the number of pieces with the least waves x tiles. A block's start
    // and end count as 3 tiles, the join as 2 and its traffic (every piece's O in fp32,
    // written and read) at 16 MB in the time of a tile (2.5 us).
    const long long piece_bytes = static_cast<long long>(t->total_q) * Hq * c->D * 8;
    long long best = -1;
    for (long long n = 1; n <= 16 && n <= nt; ++n) {
      const long long per = (nt + n - 1) / n;
      const long long waves = (units * n + num_sms() - 1) / num_sms();
      const long long cost = 100 * waves * (per + 3) + (n > 1 ? 200 + n * piece_bytes / 160000 : 0);
      if (best < 0 || cost < best) {
        best = cost;
        chunk = per;
      }
    }
    // fewer units than SMs: the SMs left over take the ends of all ranges, in as many
    // rounds as it takes, while the units' own blocks do the rest
    const long long spare = num_sms() - units;
    if (spare > 0) {
      const long long rounds = (units + spare - 1) / spare;
      const long long end = (nt + 3 - 3 * rounds) / (rounds + 1);
      if (end > 0 && 100 * (nt - end + 3) + 200 + 2 * piece_bytes / 160000 < best) {
        chunk = end;
        chunk0 = nt - end;
      }
    }
  }
  a.chunk = static_cast<int>(chunk < nt ? chunk : nt);
  a.chunk0 = static_cast<int>(chunk0 > 0 ? chunk0 : a.chunk);
  a.nsplit = chunk0 > 0 ? 2 : static_cast<int>((nt + a.chunk - 1) / a.chunk);
  // where all blocks run at once latency counts; in several waves a cluster's blocks wait
  // for one another's places (batch of 48: 95 us clustered, 91 us not)
  a.clustered = !a.tiles && a.nsplit > 1 && a.nsplit <= 8 &&
                units * a.nsplit <= decode_blocks(c, a.row_tile) * static_cast<long long>(num_sms());
  return a;
}

size_t paged_workspace(const AttnPlan& a, const ll_token_batch* t, int Hq, int D) {
  if (a.nsplit <= 1 || a.clustered) return 0;
  return align256(static_cast<size_t>(t->total_q) * Hq * a.nsplit * D * sizeof(float)) +
         align256(static_cast<size_t>(t->total_q) * Hq * a.nsplit * sizeof(float2));
}

// A window shortens every range to itself, the positions of a unit's rows and the sinks
// (a prefix may be of any length). The workspace is sized without it, so its plan is
// taken where it needs no more.
AttnPlan plan_attention(const ll_paged_cache* c, const ll_token_batch* t, int Hq, const ll_score_desc* sc) {
  const AttnPlan a = plan_for_span(c, t, Hq, 0);
  if (sc->window == 0 || sc->prefix_len != nullptr) return a;
  const long long rows = 256 / (Hq / c->H) + 2;
  const AttnPlan w = plan_for_span(c, t, Hq, static_cast<long long>(sc->window) + sc->n_sink + rows);
  return paged_workspace(w, t, Hq, c->D) <= paged_workspace(a, t, Hq, c->D) ? w : a;
}

template <class TR, int MODS>
ll_status launch_paged_decode(const ll::PagedAttnParams& p, cudaStream_t s) {
  auto kern = ll::paged_decode_kernel<TR, MODS>;
  static std::atomic<unsigned long long> done{0};
  ll_status st = allow_smem(kern, TR::SMEM, done);
  if (st != LL_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.nsplit * p.row_tiles, p.pool.H, p.batch.B);
  cfg.blockDim = dim3(TR::THREADS);
  cfg.dynamicSmemBytes = TR::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.nsplit;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.clustered ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kern, p);
  return check_launch("paged_decode_kernel");
}

template <class TR, int MODS>
ll_status launch_paged_prefill(const ll::PagedAttnParams& p, cudaStream_t s) {
  auto kern = ll::paged_prefill_kernel<TR, MODS>;
  static std::atomic<unsigned long long> done{0};
  ll_status st = allow_smem(kern, TR::SMEM, done);
  if (st != LL_OK) return st;
  kern<<<dim3(p.pool.H, p.batch.B, p.row_tiles * p.nsplit), TR::THREADS, TR::SMEM, s>>>(p);
  return check_launch("paged_prefill_kernel");
}

template <int D, bool E4M3, int MODS>
ll_status launch_paged(const AttnPlan& plan, const ll::PagedAttnParams& p, cudaStream_t s) {
  if (plan.tiles) return launch_paged_prefill<ll::PrefillTraits<D, E4M3>, MODS>(p, s);
  return plan.row_tile == 8 ? launch_paged_decode<ll::DecodeTraits<D, E4M3, 8>, MODS>(p, s)
                            : launch_paged_decode<ll::DecodeTraits<D, E4M3, 16>, MODS>(p, s);
}

template <int D, bool E4M3>
ll_status launch_paged(const AttnPlan& plan, const ll::PagedAttnParams& p, cudaStream_t s) {
  const bool capped = p.sc.cap2 > 0.f, biased = p.sc.biased != 0;
  if (capped && biased) return launch_paged<D, E4M3, ll::kCapped | ll::kBiased>(plan, p, s);
  if (capped) return launch_paged<D, E4M3, ll::kCapped>(plan, p, s);
  if (biased) return launch_paged<D, E4M3, ll::kBiased>(plan, p, s);
  return launch_paged<D, E4M3, 0>(plan, p, s);
}

// The join starts while the pieces' kernel drains and waits for its end on the
// device, which hides most of a launch.
template <int D>
ll_status launch_paged_join(const ll::PagedAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch.max_q) * p.Hq, p.batch.B);
  cfg.blockDim = dim3(ll::kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, ll::paged_join_kernel<D>, p);
  return check_launch("paged_join_kernel");
}

}  // namespace

extern "C" {

ll_status ll_token_rope_init(ll_token_rope_desc* desc, int rot_dim, int layout, double theta0, double scale,
                             double original_len, double beta_fast, double beta_slow, double amplitude) {
  g_last_error.clear();
  if (desc == nullptr) return fail(LL_ERR_INVALID_ARG, "desc is NULL");
  if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > 2 * LL_MAX_TOKEN_PAIRS)
    return fail(LL_ERR_INVALID_ARG, "rot_dim = %d must be a multiple of 16 in [16, %d]", rot_dim, 2 * LL_MAX_TOKEN_PAIRS);
  if (layout != LL_ROPE_INTERLEAVED && layout != LL_ROPE_HALF)
    return fail(LL_ERR_INVALID_ARG, "unknown rope layout %d", layout);
  if (!(theta0 > 1.0) || !std::isfinite(theta0))
    return fail(LL_ERR_INVALID_ARG, "rope theta0 must be a finite value > 1");
  if (!(scale > 0.0 && scale <= 1.0)) return fail(LL_ERR_INVALID_ARG, "rope scale must lie in (0, 1]");
  if (!(original_len >= 0.0) || !std::isfinite(original_len))
    return fail(LL_ERR_INVALID_ARG, "rope original_len must be a finite value >= 0");
  if (original_len > 0.0 && !(beta_slow >= 0.0 && beta_fast > beta_slow && std::isfinite(beta_fast)))
    return fail(LL_ERR_INVALID_ARG, "need 0 <= beta_slow < beta_fast, finite");
  if (!std::isfinite(amplitude) || !std::isfinite(static_cast<float>(amplitude)))
    return fail(LL_ERR_INVALID_ARG, "rope amplitude must be finite");
  std::memset(desc, 0, sizeof(*desc));
  desc->rot_dim = rot_dim;
  desc->layout = layout;
  desc->amplitude = static_cast<float>(amplitude);
  constexpr double kTwoPi = 6.283185307179586476925;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(theta0, -2.0 * i / rot_dim);
    double keep = 0.0;
    if (original_len > 0.0) {
      keep = (original_len * w / kTwoPi - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
    }
    // w <= 1, so the turn per position is below 1/6; the double's 53 bits put the
    // angle of position 2^31 within 2^-24 of a turn
    desc->turns[i] = static_cast<uint64_t>(std::ldexp(w * (keep + (1.0 - keep) * scale) / kTwoPi, 64));
  }
  return LL_OK;
}

ll_status ll_token_rope_apply(const void* x, long long x_stride, void* out, long long out_stride, ll_dtype dtype,
                              const int32_t* positions, int T, int H, int D, const ll_token_rope_desc* rope,
                              int transpose, void* stream) {
  g_last_error.clear();
  if (dtype != LL_F32 && dtype != LL_BF16) return fail(LL_ERR_INVALID_ARG, "dtype must be F32 or BF16");
  if (rope == nullptr || positions == nullptr) return fail(LL_ERR_INVALID_ARG, "rope and positions must be non-NULL");
  if (!aligned4(positions)) return fail(LL_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if (T < 0 || H < 1 || D < 16 || D % 16 != 0)
    return fail(LL_ERR_INVALID_ARG, "need T >= 0, H >= 1 and D a multiple of 16 (T=%d H=%d D=%d)", T, H, D);
  if (D > 1024 || static_cast<long long>(H) * D >= (1ll << 24))
    return fail(LL_ERR_UNSUPPORTED, "D = %d exceeds 1024 or H * D reaches 2^24", D);
  ll_status st = check_rows("x", x, x_stride, H, D);
  if (st != LL_OK) return st;
  if ((st = check_rows("out", out, out_stride, H, D)) != LL_OK) return st;
  ll::TokenRopeParams p;
  if ((st = make_token_rope(rope, D, transpose, &p.rope)) != LL_OK) return st;
  if (T == 0) return LL_OK;
  p.x = x;
  p.out = out;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.positions = positions;
  p.T = T;
  p.H = H;
  p.D = D;
  // one token per block while that leaves SMs idle; from there on up to 8 tokens,
  // and no more than three units per thread
  const int per_token = H * (D / 16);
  int tokens = 3 * ll::kTokenRopeThreads / per_token;
  const int fill = T / (4 * num_sms());
  tokens = tokens < fill ? tokens : fill;
  p.tokens = tokens < 1 ? 1 : (tokens > 8 ? 8 : tokens);
  const int grid = (T - 1) / p.tokens + 1;
  const size_t smem = ll::turn_table_bytes(p.tokens, p.rope.rot / 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == LL_F32)
    ll::token_rope_kernel<float><<<grid, ll::kTokenRopeThreads, smem, s>>>(p);
  else
    ll::token_rope_kernel<__nv_bfloat16><<<grid, ll::kTokenRopeThreads, smem, s>>>(p);
  return check_launch("token_rope_kernel");
}

ll_status ll_paged_append(const ll_paged_cache* cache, const ll_token_batch* batch, const void* k, long long k_stride,
                          const void* v, long long v_stride, ll_dtype in_dtype, const ll_token_rope_desc* rope,
                          void* stream) {
  g_last_error.clear();
  ll_status st = check_paged_cache(cache);
  if (st != LL_OK) return st;
  if ((st = check_batch(batch)) != LL_OK) return st;
  if (in_dtype != LL_BF16) return fail(LL_ERR_INVALID_ARG, "k and v must be BF16");
  if ((st = check_rows("k", k, k_stride, cache->H, cache->D)) != LL_OK) return st;
  if ((st = check_rows("v", v, v_stride, cache->H, cache->D)) != LL_OK) return st;
  ll::PagedAppendParams p{};
  if ((st = make_token_rope(rope, cache->D, 0, &p.rope)) != LL_OK) return st;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.pool = to_pool(cache);
  p.batch = to_batch(batch, cache->page_size);
  const int max_q = p.batch.max_q;
  if (max_q == 0) return LL_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pairs = p.rope.rot / 2, ps = cache->page_size;
  if (cache->dtype == LL_BF16) {
    // tokens per block: a thread's share of them in flight, while that leaves 4 blocks to an SM
    const int per_token = cache->H * (cache->D / 16);
    const int abreast = per_token < ll::kPagedAppendThreads ? ll::kPagedAppendThreads / per_token : 1;
    const long long fill = static_cast<long long>(max_q) * batch->B / (4 * num_sms());
    int tokens = abreast * ll::kAppendAhead;
    if (tokens > ll::kAppendMaxTokens) tokens = ll::kAppendMaxTokens;
    p.tokens = tokens < fill ? tokens : (fill < 1 ? 1 : static_cast<int>(fill));
    ll::paged_append_bf16_kernel<<<dim3((max_q - 1) / p.tokens + 1, batch->B), ll::kPagedAppendThreads,
                                   ll::turn_table_bytes(p.tokens, pairs), s>>>(p);
    return check_launch("paged_append_bf16_kernel");
  }
  const int units = ps * (cache->D / 16);  // 16-element units of a page and head: 64 to 1024
  const int side = units < 128 ? 128 / units : 1;
  // pages that max_q tokens can touch, wherever the first of them stands
  const int touched = (max_q - 1) / ps + ((max_q - 1) % ps != 0 ? 2 : 1);
  // heads per block: doubled while that divides them and leaves 4 blocks to an SM
  const long long pages = static_cast<long long>(touched) * batch->B;
  p.heads = side;
  while (cache->H % (2 * p.heads) == 0 && pages * (cache->H / (2 * p.heads)) >= 4 * num_sms()) p.heads *= 2;
  static std::atomic<unsigned long long> done{0};
  st = allow_smem(ll::paged_append_e4m3_kernel, static_cast<int>(ll::turn_table_bytes(128, LL_MAX_TOKEN_PAIRS)), done);
  if (st != LL_OK) return st;
  ll::paged_append_e4m3_kernel<<<dim3(touched, batch->B, (cache->H + p.heads - 1) / p.heads), side * units,
                                 ll::turn_table_bytes(max_q < ps ? max_q : ps, pairs), s>>>(p);
  return check_launch("paged_append_e4m3_kernel");
}

size_t ll_paged_attention_workspace_bytes(const ll_paged_cache* cache, const ll_token_batch* batch, int Hq) {
  if (check_paged_cache(cache) != LL_OK || check_batch(batch) != LL_OK || Hq < 1 || Hq % cache->H != 0 ||
      Hq > LL_MAX_TOKEN_HEADS)
    return 0;
  return paged_workspace(plan_for_span(cache, batch, Hq, 0), batch, Hq, cache->D);
}

ll_status ll_paged_attention(const void* q, long long q_stride, ll_dtype q_dtype, int Hq, const ll_paged_cache* cache,
                             const ll_token_batch* batch, const ll_token_rope_desc* rope, const ll_score_desc* scores,
                             void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  ll_status st = check_paged_cache(cache);
  if (st != LL_OK) return st;
  if ((st = check_batch(batch)) != LL_OK) return st;
  if (q_dtype != LL_BF16) return fail(LL_ERR_INVALID_ARG, "q must be BF16");
  if (Hq < 1 || Hq % cache->H != 0)
    return fail(LL_ERR_INVALID_ARG, "Hq = %d must be a positive multiple of the cache's H = %d", Hq, cache->H);
  if (Hq > LL_MAX_TOKEN_HEADS) return fail(LL_ERR_UNSUPPORTED, "Hq = %d exceeds %d", Hq, LL_MAX_TOKEN_HEADS);
  if ((st = check_rows("q", q, q_stride, Hq, cache->D)) != LL_OK) return st;
  if (out == nullptr || !aligned16(out)) return fail(LL_ERR_INVALID_ARG, "out must be non-NULL and 16-byte aligned");
  if (!aligned4(lse)) return fail(LL_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  ll::PagedAttnParams p{};
  if ((st = make_token_rope(rope, cache->D, 0, &p.rope)) != LL_OK) return st;
  const ll_score_desc plain = {};
  const ll_score_desc* sc = scores ? scores : &plain;
  if (!(sc->softmax_scale >= 0.f) || !std::isfinite(sc->softmax_scale))
    return fail(LL_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  if (!(sc->soft_cap >= 0.f) || !std::isfinite(sc->soft_cap))
    return fail(LL_ERR_INVALID_ARG, "soft_cap must be finite and >= 0");
  if (sc->window < 0 || sc->n_sink < 0) return fail(LL_ERR_INVALID_ARG, "window and n_sink must be >= 0");
  if (!aligned4(sc->prefix_len)) return fail(LL_ERR_INVALID_ARG, "prefix_len must be 4-byte aligned");
  const float scale = sc->softmax_scale > 0.f ? sc->softmax_scale : 1.0f / std::sqrt(static_cast<float>(cache->D));
  p.sc.pre = sc->soft_cap > 0.f ? scale / sc->soft_cap : scale * ll::kLog2e;
  p.sc.cap2 = sc->soft_cap * ll::kLog2e;
  if (!std::isfinite(p.sc.pre) || !std::isfinite(p.sc.cap2))
    return fail(LL_ERR_INVALID_ARG, "softmax_scale (over soft_cap) or soft_cap leaves fp32's range");
  p.sc.window = sc->window;
  p.sc.n_sink = sc->n_sink;
  p.sc.prefix_len = sc->prefix_len;
  if (sc->slopes != nullptr) {
    p.sc.biased = 1;
    for (int h = 0; h < Hq; ++h) {
      if (!std::isfinite(sc->slopes[h])) return fail(LL_ERR_INVALID_ARG, "slopes[%d] is not finite", h);
      p.sc.slope2[h] = sc->slopes[h] * ll::kLog2e;
      if (!std::isfinite(p.sc.slope2[h])) return fail(LL_ERR_INVALID_ARG, "slopes[%d] leaves fp32's range", h);
    }
  }
  const AttnPlan plan = plan_attention(cache, batch, Hq, sc);
  const size_t need = paged_workspace(plan, batch, Hq, cache->D);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(LL_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, need);
  if (need > 0 && !aligned16(workspace)) return fail(LL_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.Hq = Hq;
  p.group = Hq / cache->H;
  p.pool = to_pool(cache);
  p.batch = to_batch(batch, cache->page_size);
  p.row_tile = plan.row_tile;
  p.key_tile = plan.key_tile;
  p.row_tiles = plan.row_tiles;
  p.chunk = plan.chunk;
  p.chunk0 = plan.chunk0;
  p.nsplit = plan.nsplit;
  p.clustered = plan.clustered;
  if (need > 0) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(
        static_cast<char*>(workspace) +
        align256(static_cast<size_t>(batch->total_q) * Hq * plan.nsplit * cache->D * sizeof(float)));
  }
  if (p.batch.max_q == 0) return LL_OK;
  if (static_cast<long long>(p.nsplit) * p.row_tiles > INT_MAX || static_cast<long long>(p.batch.max_q) * Hq > INT_MAX)
    return fail(LL_ERR_UNSUPPORTED, "the call needs more than 2^31 - 1 blocks");
  if (plan.tiles && static_cast<long long>(p.row_tiles) * p.nsplit > 65535)
    return fail(LL_ERR_UNSUPPORTED, "max_q x Hq / H = %lld exceeds 256 x 65535 rows",
                static_cast<long long>(p.batch.max_q) * p.group);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == LL_FP8_E4M3;
  if (cache->D == 128)
    st = e4m3 ? launch_paged<128, true>(plan, p, s) : launch_paged<128, false>(plan, p, s);
  else
    st = e4m3 ? launch_paged<64, true>(plan, p, s) : launch_paged<64, false>(plan, p, s);
  if (st != LL_OK || need == 0) return st;
  return cache->D == 128 ? launch_paged_join<128>(p, s) : launch_paged_join<64>(p, s);
}

}  // extern "C"
