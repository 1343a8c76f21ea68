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
  int B, max_pages, total_q, max_q;
  int max_key;  // keys that may exist: min(max_kv, max_pages * page_size, 2^31 - 257)
};

// Sequence b with everything the device arrays say brought within bounds (32-bit
// throughout: positions lie in (-2^31, 2^31 - 1)).
struct SeqView {
  int q0, nq;     // rows [q0, q0 + nq) of the token tensors are processed
  int first_pos;  // position of row q0 (may be negative: such rows stand before the first key)
  int len;        // keys [0, len) exist
};

__device__ __forceinline__ SeqView seq_view(const TokenBatch& t, int b) {
  const int a = t.q_start[b], e = t.q_start[b + 1], kv = max(t.kv_len[b], 0);
  SeqView s;
  s.q0 = min(max(a, 0), t.total_q);
  const int rows = max(e, s.q0) - s.q0;
  s.first_pos = kv - rows;
  s.nq = min(min(rows, t.max_q), t.total_q - s.q0);
  s.len = min(kv, t.max_key);
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

// The angle of position `pos` in units of 2^-32 turns: the upper half of pos * turn
// modulo 2^64. Exact but for the 2^-32 cut off, so a far position costs no accuracy (a
// product of an fp32 position and frequency would be off by 0.03 rad at position 10^6).
__device__ __forceinline__ uint32_t turned(int pos, unsigned long long turn) {
  const uint32_t p = static_cast<uint32_t>(pos), lo = static_cast<uint32_t>(turn), hi = static_cast<uint32_t>(turn >> 32);
  return __umulhi(p, lo) + p * hi - (pos < 0 ? lo : 0u);  // p is pos + 2^32 where pos < 0
}

// (cos, sin) of that angle, times the amplitude. The nearest quarter turn is taken off
// in integers, so the rest (at most an eighth of a turn, y <= pi / 4) keeps all of
// fp32's bits; there the Taylor polynomials to y^9 and y^10 are within 2e-9.
__device__ __forceinline__ float2 turn_of(const TokenRope& r, int pos, unsigned long long turn) {
  const uint32_t t = turned(pos, turn);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float y = static_cast<float>(static_cast<int>(t - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = y * y;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(z, s, 1.f / 120.f);
  s = fmaf(z, s, -1.f / 6.f);
  s = fmaf(y * z, s, y);
  float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(z, c, -1.f / 720.f);
  c = fmaf(z, c, 1.f / 24.f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float u = (quarter & 1 ? s : c) * r.amp, v = (quarter & 1 ? c : s) * (r.amp * r.sign);
  return make_float2((quarter + 1) & 2 ? -u : u, quarter & 2 ? -v : v);  // quarters 1, 2; quarters 2, 3
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
  for (int t = threadIdx.x >> 5; t < nt; t += blockDim.x >> 5) {
    const int pos = position_of(t);
    for (int i = threadIdx.x & 31; i < tab.pairs; i += 32)
      cs[t * (tab.pairs + 8) + (i & 7) * tab.step + (i >> 3)] = turn_of(r, pos, s_turns[i]);
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
  const int per_head = p.D >> 4, per_token = p.H * per_head;
  const int items = nt * per_token;
  // a unit's place, and its two chunks
  struct Unit {
    int t, c, lo, hi;
    const T* src;
    T* dst;
  };
  auto unit_of = [&](int i) {
    Unit u;
    u.t = i / per_token;
    const int r = i - u.t * per_token, h = r / per_head;
    u.c = r - h * per_head;
    item_chunks(p.rope, u.c, u.lo, u.hi);
    u.src = static_cast<const T*>(p.x) + (t0 + u.t) * p.x_stride + h * p.D;
    u.dst = static_cast<T*>(p.out) + (t0 + u.t) * p.out_stride + h * p.D;
    return u;
  };
  float a[8], b[8];
  auto load = [&](const Unit& u) {
    load_chunk8<T>(u.src + u.lo * 8, a);
    load_chunk8<T>(u.src + u.hi * 8, b);
  };
  // the first unit's loads are in flight while the table is made
  int i = threadIdx.x;
  Unit u{};
  if (i < items) load(u = unit_of(i));
  const TurnTable tab = make_turn_table(p.rope, s_cs, nt, [&](int t) { return p.positions[t0 + t]; });
  while (i < items) {
    if (u.c < (p.rope.rot >> 4)) rotate_item(p.rope, a, b, tab.unit(u.t, u.c), tab.step);
    store_chunk8<T>(u.dst + u.lo * 8, a);
    store_chunk8<T>(u.dst + u.hi * 8, b);
    i += blockDim.x;
    if (i < items) load(u = unit_of(i));
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
  int n_pages, page_size, page_shift, H, D;  // page_size = 1 << page_shift
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

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// BF16 pool: a block takes `tokens` tokens of one sequence, all heads. A thread keeps
// its head and chunks and goes from token to token, kAppendAhead of them in flight, so
// nothing is divided or looked up per unit (3889 tokens of 12 heads of 128: 14.7 us a
// call, 10.9 replayed out of a graph; floor 7.3).
constexpr int kAppendAhead = 2, kAppendMaxTokens = 32;

__global__ void __launch_bounds__(kPagedAppendThreads) paged_append_bf16_kernel(const PagedAppendParams p) {
  extern __shared__ float2 s_cs[];
  __shared__ long long s_row[kAppendMaxTokens];  // first row of the token's page, all heads', plus its row; -1: none
  const int b = blockIdx.y;
  const SeqView s = seq_view(p.batch, b);
  const int i0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, s.nq - i0);
  if (nt <= 0) return;
  const int D = p.pool.D, H = p.pool.H, shift = p.pool.page_shift;
  for (int t = threadIdx.x; t < nt; t += blockDim.x) {
    const int pos = s.first_pos + i0 + t;
    int page = -1;
    if (pos >= 0 && pos >> shift < p.batch.max_pages) page = page_of(p.batch, b, pos >> shift, p.pool.n_pages);
    s_row[t] = page < 0 ? -1 : (static_cast<long long>(page) * H << shift) + (pos & (p.pool.page_size - 1));
  }
  const int log_units = D == 128 ? 3 : 2;  // units of 16 elements in a head
  const int per_token = H << log_units;
  const int abreast = per_token < kPagedAppendThreads ? kPagedAppendThreads / per_token : 1;  // tokens at a time
  const int t_mine = threadIdx.x / per_token, u0 = threadIdx.x - t_mine * per_token;
  const TurnTable tab = make_turn_table(p.rope, s_cs, nt, [&](int t) { return s.first_pos + i0 + t; });
  if (t_mine >= abreast) return;
  for (int u = u0; u < per_token; u += kPagedAppendThreads) {
    const int h = u >> log_units, c = u & ((1 << log_units) - 1);
    int lo, hi;
    item_chunks(p.rope, c, lo, hi);
    const bool turns = c < (p.rope.rot >> 4);
    const __nv_bfloat16* kr = p.k + static_cast<size_t>(s.q0 + i0) * p.k_stride + h * D;
    const __nv_bfloat16* vr = p.v + static_cast<size_t>(s.q0 + i0) * p.v_stride + h * D;
    __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(p.pool.k);
    __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(p.pool.v);
    for (int t0 = t_mine; t0 < nt; t0 += abreast * kAppendAhead) {
      uint4 raw[kAppendAhead][4];
#pragma unroll
      for (int k = 0; k < kAppendAhead; ++k) {
        const int t = t0 + k * abreast;
        if (t < nt) {
          raw[k][0] = *reinterpret_cast<const uint4*>(kr + t * p.k_stride + lo * 8);
          raw[k][1] = *reinterpret_cast<const uint4*>(kr + t * p.k_stride + hi * 8);
          raw[k][2] = *reinterpret_cast<const uint4*>(vr + t * p.v_stride + lo * 8);
          raw[k][3] = *reinterpret_cast<const uint4*>(vr + t * p.v_stride + hi * 8);
        }
      }
#pragma unroll
      for (int k = 0; k < kAppendAhead; ++k) {
        const int t = t0 + k * abreast;
        if (t >= nt || s_row[t] < 0) continue;
        const size_t at = static_cast<size_t>(s_row[t] + (static_cast<long long>(h) << shift)) * D;
        float x[8], y[8];
        unpack8(raw[k][0], x);
        unpack8(raw[k][1], y);
        if (turns) rotate_item(p.rope, x, y, tab.unit(t, c), tab.step);
        store_chunk8<__nv_bfloat16>(kd + at + lo * 8, x);
        store_chunk8<__nv_bfloat16>(kd + at + hi * 8, y);
        *reinterpret_cast<uint4*>(vd + at + lo * 8) = raw[k][2];
        *reinterpret_cast<uint4*>(vd + at + hi * 8) = raw[k][3];
      }
    }
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

// |x|, 0 for an infinity or NaN
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// E4M3 codes of x * inv: to nearest even, saturating at +-448 (NaN stays NaN).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  const uint64_t inv2 = f2_pack(inv, inv);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(f2_pack(x[2 * i], x[2 * i + 1]), inv2), y[2 * i], y[2 * i + 1]);
  return make_uint2(encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7]));
}

// 1 / s for a scale, 0 for 0. A power of two's is one subtraction of exponents.
__device__ __forceinline__ float inverse_scale(float s) {
  const uint32_t u = __float_as_uint(s);
  if ((u & 0x807FFFFFu) == 0 && u >= 0x00800000u && u <= 0x7E800000u) return __uint_as_float(0x7F000000u - u);
  return s > 0.f ? 1.0f / s : 0.f;
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

// The largest |x| of eight bf16 values, NaN left out.
__device__ __forceinline__ __nv_bfloat162 bf16_amax(const uint4& u, __nv_bfloat162 a) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) a = __hmax2(a, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  return a;
}

// 8-bit pool: a block takes one page of one sequence and `heads` heads of it, `side`
// of them at a time, a thread per unit of 16 elements of a head's K and V. They stay in
// registers between the maximum over the page and the codes, so each is read once;
// the next heads' loads are issued before this round's barrier. The angles are computed
// once for all heads of a block. Measured (8800 tokens, 8 heads of 128, pages of 64): a
// block per head, 65 us; angles shared but two units per thread, so that registers left
// one block per SM, 42 us; as here 20.7 us, floor 8.2.
__global__ void __launch_bounds__(kPagedAppendMaxThreads, 1) paged_append_e4m3_kernel(const PagedAppendParams p) {
  extern __shared__ float2 s_cs[];
  __shared__ uint32_t s_max[2][2][kPagedAppendMaxThreads / 32];  // [parity][K, V][warp]: bits of the maximum
  const int b = blockIdx.y, ps = p.pool.page_size, D = p.pool.D, H = p.pool.H;
  const SeqView s = seq_view(p.batch, b);
  // page number within the sequence, and the rows of it that are new
  const int beg = max(s.first_pos, 0), end = s.first_pos + s.nq;
  const int pg = (beg >> p.pool.page_shift) + blockIdx.x;
  if (pg >= p.batch.max_pages || pg > (end - 1) >> p.pool.page_shift || end <= beg) return;
  const int n0 = max(beg - pg * ps, 0), n1 = min(end - pg * ps, ps);
  const int page = page_of(p.batch, b, pg, p.pool.n_pages);
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
  const int row = s.q0 + (pg * ps - s.first_pos) + slot;  // of the token tensors, where fresh
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
      // an infinity shows in the maximum (NaN never does): only then it is looked for
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmax3(a, fabsf(x[e]), fabsf(y[e]));
      const __nv_bfloat162 vm = bf16_amax(v1, bf16_amax(v0, __floats2bfloat162_rn(0.f, 0.f)));
      float av = fmaxf(__low2float(vm), __high2float(vm));
      if (fmaxf(a, av) > 3.402823466e38f) {
        float z[8], q[8];
        unpack8(v0, z);
        unpack8(v1, q);
        a = av = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a = fmax3(a, finite_abs(x[e]), finite_abs(y[e]));
          av = fmax3(av, finite_abs(z[e]), finite_abs(q[e]));
        }
      }
      amax[0] = __float_as_uint(a);
      amax[1] = __float_as_uint(av);
    }
    load(h + side);
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // non-negative floats order as integers
      amax[w] = __reduce_max_sync(0xffffffffu, amax[w]);
      if ((threadIdx.x & 31) == 0) s_max[parity][w][threadIdx.x >> 5] = amax[w];
    }
    __syncthreads();  // one per round: the next round writes the other parity
    if (!live) continue;  // a whole warp
    float scale[2], inv[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int lane = threadIdx.x & 31;  // of the head's warps (at most 32), one each
      const uint32_t m =
          __reduce_max_sync(0xffffffffu, lane < units >> 5 ? s_max[parity][w][slot_h * (units >> 5) + lane] : 0u);
      scale[w] = fmaxf(was[w], two_power_scale(__uint_as_float(m)));
      inv[w] = inverse_scale(scale[w]);
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
