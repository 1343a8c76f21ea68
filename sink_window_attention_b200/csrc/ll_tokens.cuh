// ll_tokens.cuh — streams of single tokens: the batch descriptor as the kernels
// see it, rotary positions of token tensors, and the append to a paged pool.
#pragma once

#include <cuda_fp16.h>

#include "ll_common.cuh"
#include "ll_rope_append.cuh"

namespace ll {

// ---------------------------------------------------------------------------
// Which tokens a call works on
// ---------------------------------------------------------------------------
struct TokenBatch {
  const int* q_start;
  const int* kv_len;
  const int* page_table;
  int B, max_pages, total_q, max_q, max_kv;
};

// Sequence b with everything the device arrays say brought within bounds.
struct SeqView {
  int q0, nq;           // rows [q0, q0 + nq) of the token tensors are processed
  long long first_pos;  // position of row q0 (may be negative: such rows stand before the first key)
  int len;              // keys [0, len) exist
};

__device__ __forceinline__ SeqView seq_view(const TokenBatch& t, int b, int page_size) {
  SeqView s;
  const long long a = t.q_start[b], e = t.q_start[b + 1], kv = t.kv_len[b];
  const long long rows = e > a ? e - a : 0;
  s.q0 = static_cast<int>(a < 0 ? 0 : (a > t.total_q ? t.total_q : a));
  s.first_pos = kv - rows + (s.q0 - a);
  long long n = rows - (s.q0 - a);
  n = n < t.max_q ? n : t.max_q;
  n = n < t.total_q - s.q0 ? n : t.total_q - s.q0;
  s.nq = static_cast<int>(n > 0 ? n : 0);
  const long long cap = static_cast<long long>(t.max_pages) * page_size;
  long long len = kv < t.max_kv ? kv : t.max_kv;
  len = len < cap ? len : cap;
  s.len = static_cast<int>(len > 0 ? len : 0);
  return s;
}

// Page of token j of sequence b, or -1 where the table names none.
__device__ __forceinline__ int page_of(const TokenBatch& t, int b, int page, int n_pages) {
  const int p = t.page_table[static_cast<size_t>(b) * t.max_pages + page];
  return p >= 0 && p < n_pages ? p : -1;
}

// ---------------------------------------------------------------------------
// Rotation
// ---------------------------------------------------------------------------
constexpr int kMaxTokenPairs = 64;

struct TokenRope {
  int rot;     // rotated elements of a head; 0: no rotation
  int half;    // pairs (i, i + rot/2) instead of (2i, 2i + 1)
  float amp;
  float sign;  // -1: the transposed rotation
  unsigned long long turns[kMaxTokenPairs];
};

// (cos, sin) of a pair at position `pos`, times the amplitude. The angle in turns is
// pos * turn modulo 2^64: exact, so a far position costs no accuracy (a
// product of an fp32 position and frequency would be off by 0.03 rad at
// position 10^6). The nearest quarter turn is taken off in integers, so the rest
// (at most an eighth of a turn) keeps all of fp32's bits.
__device__ __forceinline__ float2 turn_of(const TokenRope& r, long long pos, unsigned long long turn) {
  const uint32_t t = static_cast<uint32_t>((static_cast<unsigned long long>(pos) * turn) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int>(t - (quarter << 30))) * 4.656612873077393e-10f;  // half turns
  float s, c;
  sincospif(a, &s, &c);
  float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  if ((quarter + 1) & 2) x = -x;  // quarters 1 and 2
  if (quarter & 2) y = -y;        // quarters 2 and 3
  return make_float2(x * r.amp, y * r.amp * r.sign);
}

// The unit that the rotating kernels work in: 16 elements of a head, pairs
// 8c .. 8c + 7. In the half layout they are the 8-element chunks c of the lower
// and of the upper half; else (and past rot) the neighbouring chunks 2c, 2c + 1.
__device__ __forceinline__ void item_chunks(const TokenRope& r, int c, int& lo, int& hi) {
  const int pairs8 = r.rot >> 4;
  if (r.half && c < pairs8) {
    lo = c;
    hi = c + pairs8;
  } else {
    lo = 2 * c;
    hi = 2 * c + 1;
  }
}

// cs: (cos, sin) of the unit's 8 pairs, `step` apart.
__device__ __forceinline__ void rotate_item(const TokenRope& r, float (&a)[8], float (&b)[8], const float2* cs, int step) {
  if (r.half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = cs[i * step];
      const float x = a[i], y = b[i];
      a[i] = x * t.x - y * t.y;
      b[i] = x * t.y + y * t.x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = cs[i * step], u = cs[(4 + i) * step];
      float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * t.x - y * t.y;
      a[2 * i + 1] = x * t.y + y * t.x;
      x = b[2 * i];
      y = b[2 * i + 1];
      b[2 * i] = x * u.x - y * u.y;
      b[2 * i + 1] = x * u.y + y * u.x;
    }
  }
}

// A block's table of (cos, sin): a row per token, pair 8c + e at [e][c], so that the
// lanes of neighbouring units read neighbouring entries, and 8 entries between rows
// for the units of the next tokens (64-byte reads straight from pair order met in the
// same banks four at a time).
struct TurnTable {
  float2* cs;
  int pairs, step;
  __device__ __forceinline__ const float2* unit(int token, int c) const { return cs + token * (pairs + 8) + c; }
};
__host__ __device__ inline size_t turn_table_bytes(int tokens, int pairs) {
  return pairs == 0 ? 0 : (static_cast<size_t>(tokens) * (pairs + 8) * sizeof(float2));
}

// Fills the table for `nt` tokens, position_of(t) giving their positions; two block
// barriers. The turns come from shared memory: as an index into the kernel's
// parameters that differs by lane each read would be served a lane at a time (that
// took three quarters of the append's time).
template <class F>
__device__ __forceinline__ TurnTable make_turn_table(const TokenRope& r, float2* cs, int nt, F&& position_of) {
  __shared__ unsigned long long s_turns[kMaxTokenPairs];
  TurnTable tab{cs, r.rot >> 1, r.rot >> 4};
  for (int i = threadIdx.x; i < tab.pairs; i += blockDim.x) s_turns[i] = r.turns[i];
  __syncthreads();
  for (int i = threadIdx.x; i < nt * tab.pairs; i += blockDim.x) {
    const int t = i / tab.pairs, j = i - t * tab.pairs;  // entry j of the row: pair 8 (j % step) + j / step
    const int e = j / tab.step, c = j - e * tab.step;
    cs[t * (tab.pairs + 8) + j] = turn_of(r, position_of(t), s_turns[c * 8 + e]);
  }
  __syncthreads();
  return tab;
}

// ---------------------------------------------------------------------------
// out[t][h] = R(positions[t]) x[t][h]
// ---------------------------------------------------------------------------
struct TokenRopeParams {
  const void* x;
  void* out;
  long long x_stride, out_stride;
  const int* positions;
  int T, H, D;
  int tokens;  // per block
  TokenRope rope;
};

constexpr int kTokenRopeThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kTokenRopeThreads) token_rope_kernel(const TokenRopeParams p) {
  extern __shared__ float2 s_cs[];
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  const TurnTable tab = make_turn_table(p.rope, s_cs, nt, [&](int t) { return static_cast<long long>(p.positions[t0 + t]); });
  const int per_head = p.D >> 4, per_token = p.H * per_head;
  const int items = nt * per_token;
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    const int t = i / per_token, r = i - t * per_token;
    const int h = r / per_head, c = r - h * per_head;
    int lo, hi;
    item_chunks(p.rope, c, lo, hi);
    const T* src = static_cast<const T*>(p.x) + (t0 + t) * p.x_stride + h * p.D;
    T* dst = static_cast<T*>(p.out) + (t0 + t) * p.out_stride + h * p.D;
    float a[8], b[8];
    load_chunk8<T>(src + lo * 8, a);
    load_chunk8<T>(src + hi * 8, b);
    if (c < (p.rope.rot >> 4)) rotate_item(p.rope, a, b, tab.unit(t, c), tab.step);
    store_chunk8<T>(dst + lo * 8, a);
    store_chunk8<T>(dst + hi * 8, b);
  }
}

// ---------------------------------------------------------------------------
// Append to the pool
// ---------------------------------------------------------------------------
struct PagedPool {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int n_pages, page_size, H, D;
};

struct PagedAppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_stride, v_stride;
  PagedPool pool;
  TokenBatch batch;
  TokenRope rope;
  int tokens;          // bf16 pool: tokens per block
  int heads;   // 8-bit pool: heads per block, a multiple of those side by side
};

constexpr int kPagedAppendThreads = 256;
constexpr int kPagedAppendMaxThreads = 1024;  // 8-bit pool: a thread per 16 elements of a page and head

// BF16 pool: a block takes `tokens` tokens of one sequence, all heads.
__global__ void __launch_bounds__(kPagedAppendThreads) paged_append_bf16_kernel(const PagedAppendParams p) {
  extern __shared__ float2 s_cs[];
  const int b = blockIdx.y;
  const SeqView s = seq_view(p.batch, b, p.pool.page_size);
  const int i0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, s.nq - i0);
  if (nt <= 0) return;
  const TurnTable tab = make_turn_table(p.rope, s_cs, nt, [&](int t) { return s.first_pos + i0 + t; });
  const int D = p.pool.D, H = p.pool.H, ps = p.pool.page_size;
  const int per_head = D >> 4, per_token = H * per_head;
  for (int i = threadIdx.x; i < nt * per_token; i += blockDim.x) {
    const int t = i / per_token, r = i - t * per_token;
    const int h = r / per_head, c = r - h * per_head;
    const long long pos = s.first_pos + i0 + t;
    if (pos < 0 || pos >= static_cast<long long>(p.batch.max_pages) * ps) continue;
    const int page = page_of(p.batch, b, static_cast<int>(pos / ps), p.pool.n_pages);
    if (page < 0) continue;
    int lo, hi;
    item_chunks(p.rope, c, lo, hi);
    const long long row = s.q0 + i0 + t;
    const __nv_bfloat16* kr = p.k + row * p.k_stride + h * D;
    const __nv_bfloat16* vr = p.v + row * p.v_stride + h * D;
    const uint4 v0 = *reinterpret_cast<const uint4*>(vr + lo * 8), v1 = *reinterpret_cast<const uint4*>(vr + hi * 8);
    float x[8], y[8];
    load_chunk8<__nv_bfloat16>(kr + lo * 8, x);
    load_chunk8<__nv_bfloat16>(kr + hi * 8, y);
    if (c < (p.rope.rot >> 4)) rotate_item(p.rope, x, y, tab.unit(t, c), tab.step);
    const size_t at = ((static_cast<size_t>(page) * H + h) * ps + static_cast<int>(pos % ps)) * D;
    __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(p.pool.k) + at;
    __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(p.pool.v) + at;
    store_chunk8<__nv_bfloat16>(kd + lo * 8, x);
    store_chunk8<__nv_bfloat16>(kd + hi * 8, y);
    *reinterpret_cast<uint4*>(vd + lo * 8) = v0;
    *reinterpret_cast<uint4*>(vd + hi * 8) = v1;
  }
}

// The smallest power of two s with 448 s >= amax, for finite amax >= 0 (0 for
// 0; at least 2^-126, so that 1 / s is finite). 448 = 1.75 * 2^8.
__device__ __forceinline__ float two_power_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased exponent of s
  return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // infinity and NaN do not set a scale
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ uint2 recode8(uint2 c, float ratio) {
  float x[8];
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  return encode8(x, ratio);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The largest finite |x| of eight bf16 values: as integers, where an exponent of all
// ones (infinity, NaN) counts as 0.
__device__ __forceinline__ uint32_t bf16_amax(const uint4& u, uint32_t a) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] << 16 & 0x7FFF0000u, hi = w[i] & 0x7FFF0000u;
    a = max(a, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
  }
  return a;
}

// 8-bit pool: a block takes one page of one sequence and `heads` heads of it, `side`
// of them at a time, a thread per unit of 16 elements of a head's K and V. They stay in
// registers between the maximum over the page and the codes, so each is read once;
// the next heads' loads are issued before this round's barrier. The angles are computed
// once for all heads of a block. Measured (8800 tokens, 8 heads of 128, pages of 64): a
// block per head, 65 us; angles shared but two units per thread, so that registers left
// one block per SM, 42 us.
__global__ void __launch_bounds__(kPagedAppendMaxThreads, 1) paged_append_e4m3_kernel(const PagedAppendParams p) {
  extern __shared__ float2 s_cs[];
  __shared__ uint32_t s_max[2][2][kPagedAppendMaxThreads / 32];  // [parity][K, V][warp]: bits of the maximum
  const int b = blockIdx.y, ps = p.pool.page_size, D = p.pool.D, H = p.pool.H;
  const SeqView s = seq_view(p.batch, b, ps);
  // page number within the sequence, and the rows of it that are new
  const long long beg = s.first_pos > 0 ? s.first_pos : 0;
  const long long end = s.first_pos + s.nq;
  const long long pg = beg / ps + blockIdx.x;
  if (pg * ps >= end || pg >= p.batch.max_pages) return;
  const int n0 = static_cast<int>((beg > pg * ps ? beg : pg * ps) - pg * ps);
  const int n1 = static_cast<int>((end < (pg + 1) * ps ? end : (pg + 1) * ps) - pg * ps);
  const int page = page_of(p.batch, b, static_cast<int>(pg), p.pool.n_pages);
  if (page < 0) return;
  const int per_head = D >> 4;
  const int units = ps * per_head;  // of a head: a multiple of 32, so a warp holds one head
  const int side = blockDim.x / units;
  const int slot_h = threadIdx.x / units, lt = threadIdx.x - slot_h * units;
  const int slot = lt / per_head, c = lt - slot * per_head;
  int lo, hi;
  item_chunks(p.rope, c, lo, hi);
  const bool fresh = slot >= n0 && slot < n1;
  const int h_end = min(H, static_cast<int>(blockIdx.z + 1) * p.heads);
  const long long row = s.q0 + (pg * ps - s.first_pos) + slot;  // of the token tensors
  const __nv_bfloat16* kr = p.k + row * p.k_stride;
  const __nv_bfloat16* vr = p.v + row * p.v_stride;
  uint4 raw[4];  // K lo, K hi, V lo, V hi
  auto load = [&](int h) {
    if (!fresh || h >= h_end) return;
    raw[0] = *reinterpret_cast<const uint4*>(kr + h * D + lo * 8);
    raw[1] = *reinterpret_cast<const uint4*>(kr + h * D + hi * 8);
    raw[2] = *reinterpret_cast<const uint4*>(vr + h * D + lo * 8);
    raw[3] = *reinterpret_cast<const uint4*>(vr + h * D + hi * 8);
  };
  load(blockIdx.z * p.heads + slot_h);
  const TurnTable tab = make_turn_table(p.rope, s_cs, n1 - n0, [&](int t) { return pg * ps + n0 + t; });
  int parity = 0;
  for (int hb = blockIdx.z * p.heads; hb < h_end; hb += side, parity ^= 1) {
    const int h = hb + slot_h;
    const bool live = h < h_end;
    const size_t scale_at = static_cast<size_t>(page) * H + (live ? h : 0);
    float was[2] = {0.f, 0.f};
    if (live && n0 > 0) {
      was[0] = p.pool.k_scale[scale_at];
      was[1] = p.pool.v_scale[scale_at];
    }
    float x[8], y[8];  // K
    const uint4 v0 = raw[2], v1 = raw[3];
    uint32_t amax[2] = {0u, 0u};
    if (live && fresh) {
      unpack8(raw[0], x);
      unpack8(raw[1], y);
      if (c < (p.rope.rot >> 4)) rotate_item(p.rope, x, y, tab.unit(slot - n0, c), tab.step);
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmax3(a, finite_abs(x[e]), finite_abs(y[e]));
      amax[0] = __float_as_uint(a);
      amax[1] = bf16_amax(v1, bf16_amax(v0, 0u));
    }
    load(h + side);
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // non-negative floats order as integers
      amax[w] = __reduce_max_sync(0xffffffffu, amax[w]);
      if ((threadIdx.x & 31) == 0) s_max[parity][w][threadIdx.x >> 5] = amax[w];
    }
    __syncthreads();  // one per round: the next round writes the other parity
    if (!live) continue;
    float scale[2], inv[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t m = 0u;
      for (int i = slot_h * (units >> 5); i < (slot_h + 1) * (units >> 5); ++i) m = max(m, s_max[parity][w][i]);
      scale[w] = fmaxf(was[w], two_power_scale(__uint_as_float(m)));
      inv[w] = scale[w] > 0.f ? 1.0f / scale[w] : 0.f;
    }
    uint8_t* kd = static_cast<uint8_t*>(p.pool.k) + scale_at * ps * D + static_cast<size_t>(slot) * D;
    uint8_t* vd = static_cast<uint8_t*>(p.pool.v) + scale_at * ps * D + static_cast<size_t>(slot) * D;
    if (fresh) {
      *reinterpret_cast<uint2*>(kd + lo * 8) = encode8(x, inv[0]);
      *reinterpret_cast<uint2*>(kd + hi * 8) = encode8(y, inv[0]);
      unpack8(v0, x);
      *reinterpret_cast<uint2*>(vd + lo * 8) = encode8(x, inv[1]);
      unpack8(v1, x);
      *reinterpret_cast<uint2*>(vd + hi * 8) = encode8(x, inv[1]);
    } else if (slot < n0) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!(scale[w] > was[w])) continue;  // the earlier tokens' codes stand
        uint2* cd = reinterpret_cast<uint2*>((w ? vd : kd) + c * 16);
        const uint2 c0 = cd[0], c1 = cd[1];
        cd[0] = recode8(c0, was[w] * inv[w]);
        cd[1] = recode8(c1, was[w] * inv[w]);
      }
    }
    if (lt == 0) {
      p.pool.k_scale[scale_at] = scale[0];
      p.pool.v_scale[scale_at] = scale[1];
    }
  }
}

}  // namespace ll
