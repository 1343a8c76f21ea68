// ll_paged_attention.cuh — attention of a ragged batch of token rows over a
// paged pool: the kernel for few rows (decode), and the one that joins the
// pieces of a split key range.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(x_j - m),
//   x = scale q.k, soft-capped, biased by distance; masked keys have no x.
#pragma once

#include <type_traits>

#include "ll_tokens.cuh"

namespace ll {

constexpr int kMaxTokenHeads = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct ScoreParams {
  float pre;     // factor on q.k: softmax_scale * (cap > 0 ? 1 / cap : log2 e)
  float cap2;    // cap * log2 e, or 0
  int window, n_sink;
  const int* prefix_len;
  int biased;
  float slope2[kMaxTokenHeads];  // slope * log2 e
};

struct PagedAttnParams {
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* out;
  float* lse;
  int Hq, group;     // query heads, and how many share a K/V head
  PagedPool pool;
  TokenBatch batch;
  TokenRope rope;
  ScoreParams sc;
  int row_tile;      // rows (token, query head of the group) of a unit
  int key_tile;      // keys per step; pieces begin at multiples of it
  int chunk;         // key tiles per piece
  int chunk0;        // and of the first piece, which may be longer
  int nsplit;        // pieces at most
  int clustered;     // decode: the nsplit blocks of a unit form a cluster, share its keys evenly and join on chip
  int row_tiles;     // units of a sequence and K/V head at most
  float* part_o;     // [total_q][Hq][nsplit][D], unnormalised
  float2* part_ml;   // [total_q][Hq][nsplit]: (max, sum), max in log2 units
};

// The keys that some row of a unit sees, as two runs of key tiles: [0, a_end)
// (prefix and sinks) and [w_beg, w_end) (window). Rows of the unit stand at
// positions p_lo .. p_hi.
struct KeyRange {
  int prefix, always, lo, upper;  // keys [0, always) and [lo, upper) are seen by some row
  int a_end, w_beg, nt;           // tiles in all
  __device__ __forceinline__ int tile(int i) const { return i < a_end ? i : i - a_end + w_beg; }
  __device__ __forceinline__ bool some_row_sees(int j) const { return (j < always) | ((j >= lo) & (j < upper)); }
};

// The first key that the window of position p reaches.
__device__ __forceinline__ int window_begin(const ScoreParams& sc, int p) {
  return sc.window > 0 && p >= sc.window ? p - sc.window + 1 : 0;
}

__device__ __forceinline__ KeyRange key_range(const ScoreParams& sc, int b, const SeqView& s, int p_lo, int p_hi,
                                              int key_tile) {
  KeyRange r;
  int prefix = sc.prefix_len ? sc.prefix_len[b] : 0;
  r.prefix = prefix < 0 ? 0 : (prefix < s.len ? prefix : s.len);
  r.upper = max(min(p_hi + 1, s.len), 0);  // keys [0, upper) stand at or before the last row
  r.lo = min(window_begin(sc, p_lo), r.upper);
  const int sink = sc.window > 0 ? (sc.n_sink < r.upper ? sc.n_sink : r.upper) : 0;
  r.always = sink > r.prefix ? sink : r.prefix;
  r.a_end = (r.always + key_tile - 1) / key_tile;
  const int wb = r.lo / key_tile;
  r.w_beg = wb > r.a_end ? wb : r.a_end;
  const int w_end = (r.upper + key_tile - 1) / key_tile;
  r.nt = r.a_end + (w_end > r.w_beg ? w_end - r.w_beg : 0);
  return r;
}

__device__ __forceinline__ bool row_sees(const ScoreParams& sc, const KeyRange& r, int len, int p, int j) {
  // bitwise, so that nothing has to be skipped
  const bool near = static_cast<unsigned>(p) - static_cast<unsigned>(j) < static_cast<unsigned>(sc.window);
  return (j < r.prefix) | ((j <= p) & (j < len) & ((sc.window == 0) | near | (j < sc.n_sink)));
}

// Positions of a unit's first and last row.
__device__ __forceinline__ void unit_positions(const PagedAttnParams& p, const SeqView& s, int r0, int& lo, int& hi) {
  const int last = min(r0 + p.row_tile, s.nq * p.group) - 1;
  lo = s.first_pos + r0 / p.group;
  hi = s.first_pos + last / p.group;
}

// Pieces of a range of nt tiles, and where one begins and ends: the host's bounds on
// ranges make nsplit enough; the last piece takes what they should have missed.
__device__ __forceinline__ int piece_count(const PagedAttnParams& p, int nt) {
  return nt <= p.chunk0 ? 1 : min(1 + (nt - p.chunk0 + p.chunk - 1) / p.chunk, p.nsplit);
}
__device__ __forceinline__ int piece_begin(const PagedAttnParams& p, int split) {
  return split == 0 ? 0 : p.chunk0 + (split - 1) * p.chunk;
}
__device__ __forceinline__ int piece_end(const PagedAttnParams& p, int split, int pieces, int nt) {
  return split == pieces - 1 ? nt : min(nt, piece_begin(p, split + 1));
}

// What a kernel is compiled for beyond a scaled product: a branch per score, or the
// cap's exponential in calls that have none, would cost more than a copy of the code.
enum : int { kCapped = 1, kBiased = 2 };

// p - j, for a bias: exact where it matters (below 2^24), never overflowing.
__device__ __forceinline__ float offset_of(int p, int j) {
  return p >= j ? static_cast<float>(static_cast<unsigned>(p) - j) : -static_cast<float>(static_cast<unsigned>(j) - p);
}

// tanh(y) = 1 - 2 / (1 + e^2y): within about 2e-7 absolute, which the cap scales (to some
// 1e-5 of a score at a cap of 64; the hardware's own tanh is off by 5e-4). Near 0 that is
// no relative precision, so where the cap is WIDE the series y - y^3/3 + 2 y^5/15 -
// 17 y^7/315 is taken below 1/4, whose rest is 1e-7 of y. Taken for every cap it would make
// capped tiles of 128 rows 132 -> 156 us (2619 tokens of 16 heads of 128, bf16 pool).
constexpr float kWideCap = 64.f;

template <bool WIDE>
__device__ __forceinline__ float tanh_accurate(float y) {
  const float far = 1.f - __fdividef(2.f, 1.f + ex2(2.f * kLog2e * y));
  if constexpr (!WIDE) return far;
  const float z = y * y;
  float q = fmaf(z, -17.f / 315.f, 2.f / 15.f);
  q = fmaf(z, q, -1.f / 3.f);
  return z < 0.0625f ? fmaf(y * z, q, y) : far;
}

// The score in log2 units from s = q.k; away: p - j.
template <int MODS, bool WIDE>
__device__ __forceinline__ float score2(const ScoreParams& sc, float s, float factor, float slope, float away) {
  float y = s * factor;
  if constexpr ((MODS & kCapped) != 0) y = sc.cap2 * tanh_accurate<WIDE>(y);
  if constexpr ((MODS & kBiased) != 0) y = fmaf(-slope, fabsf(away), y);
  return y;
}

// Runs f(std::true_type) where a cap is wide, f(std::false_type) otherwise.
template <int MODS, class F>
__device__ __forceinline__ void with_cap(const ScoreParams& sc, F&& f) {
  if ((MODS & kCapped) != 0 && sc.cap2 > kWideCap * kLog2e) f(std::true_type{});
  else f(std::false_type{});
}

// The power of two 2^e with 2^e <= a < 2^(e+1), kept within [2^-125, 2^126] (1 for 0).
__device__ __forceinline__ float power_below(float a) {
  const int e = static_cast<int>(__float_as_uint(a) >> 23);
  if (e == 0) return 1.f;
  return __uint_as_float(static_cast<uint32_t>(e < 2 ? 2 : (e > 253 ? 253 : e)) << 23);
}

// The exponent c of a V scale, kept within [-106, 126]. P enters the
// MMA as 2^(x + c - m) and the sum takes 2^-c of it, so that P stays in fp16 whatever the
// scales are. The sum is kept in units of 2^13 (8-bit pools), which centres it in fp32's
// range: 2^20 weights of 2^14 at c = -106 come to 2^127 units, one of 2^6 at c = 119 (the
// largest that bf16 values ask for) to 2^-126. Of values below some 2^-97 bits are lost.
// A zero scale's codes are zeros and ask for no c: -40 leaves the other pages' P their bits,
// and 80 binades to its own weights, which only the sum sees.
__device__ __forceinline__ int scale_exponent(float s) {
  const int e = static_cast<int>(__float_as_uint(s) >> 23 & 255u) - 127;
  return e == -127 ? -40 : (e < -106 ? -106 : (e > 126 ? 126 : e));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
template <bool E4M3>
constexpr int kSumUnit = E4M3 ? 13 : 0;  // log2

// The running reference of a row's exponents is raised where a score exceeds it by 2^8,
// so a weight is at most 2^8. bf16 weights keep their 8 bits however small they are. fp16
// ones (8-bit pools) are subnormal below 2^-14 and 0 below 2^-25, while the sum keeps them
// in fp32: behind one key with nearly all of the mass the others lost bits, and the output
// is theirs where that key's value is small. So the reference then stands 2^6 below the
// maximum: weights reach 2^14, times V's mantissa 2^15, and one of them is a normal
// down to 2^-20 of the largest, and off by at most 2^-31 of it below.
template <bool E4M3>
constexpr float kHeadroom = E4M3 ? 6.f : 0.f;

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------------------
// cp.async and mma.sync
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values, two neighbouring columns per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four E4M3 codes as two pairs of halves (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// ---------------------------------------------------------------------------
// Few rows (decode). One block: 8 or 16 rows of a sequence and K/V head against a
// piece of its keys; the block's warps take 16-key tiles in turn, each with a
// ring of its own in shared memory that cp.async keeps full, and meet once at
// the end. What bounds it is the pool's bytes: 4 warps x (STAGES - 1) tiles of K
// and V in flight per block, several blocks per SM, and few instructions per tile.
// The matrix instruction is the warp-level one (16 x 8 x 16): a tensor-memory tile
// has 128 rows, of which a decode step fills 1 to 16.
//
// Keys (and then d) are the MMA's 16 rows, the query rows its 8 columns, so 8 query
// rows waste nothing: S^T = K Q^T, then O^T = V^T P^T. The reduction index of an MMA
// may be permuted when both operands are, so neither K nor V needs a transposing load:
//  * S^T: lane (g, t) holds keys g and g + 8 and takes whole 16-byte chunks t, t + 4,
//    .. of their rows; Q's fragments use the same order of d.
//  * O^T: P leaves S^T with keys along lanes g and is turned by two 8 x 8 transposes;
//    the lane reads the V rows of keys 2t, 2t+1, 2t+8, 2t+9 at chunk g (+ 8), and
//    byte permutes pair two keys at the same d.
// One query per sequence, 8 K/V heads of 128: 4 sequences of up to 131000 keys (64 query
// heads, 8-bit pool, 701 MB) 128 us, 5.5 TB/s, 83 % of a copy's rate; 48 of 2000 to 8000
// (472 MB) 95 us, 5.0 TB/s; bf16 pool, the same 48 (945 MB) 153 us, 6.2 TB/s. With query
// rows as the MMA's 16 rows the 8-bit batch took 110 us, with a conversion per E4M3 pair
// that unpacked its operand 178 us. P in bf16 over a bf16 pool is what the matrix
// instruction takes beside V; its rounding is averaged over the keys (2.3e-3 of the
// output's norm in all, the output's own rounding 1.7e-3).
// ---------------------------------------------------------------------------
template <int D_, bool E4M3_, int ROWS_>
struct DecodeTraits {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int ROWS = ROWS_;        // 8 or 16
  static constexpr int NR = ROWS / 8;       // MMAs side by side over the rows
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * ES;
  static constexpr int CH = ROWB / 16;      // chunks per row
  static constexpr int KC = CH / 4;         // chunks of a K row per lane
  static constexpr int EPC = 16 / ES;       // elements per chunk
  static constexpr int KS = D / 16;         // MMAs over d
  static constexpr int MT = D / 16;         // MMAs over O^T's rows
  static constexpr int TILE = 16 * ROWB;
  static constexpr int NW = 4;
  static constexpr int THREADS = NW * 32;
  static constexpr int STAGES = ROWB >= 256 || ROWS == 8 ? 3 : 4;
  static constexpr int RING = NW * STAGES * 2 * TILE;
  static constexpr int QP = D + 8;          // 16-bit elements between rows of Q
  // Per SM, by shared memory and registers. 8 rows over 128-byte rows of K: 4 blocks
  // with 3 stages each read 5.6 TB/s, 3 with 4 stages 4.4, 4 with 2 stages 5.4.
  static constexpr int BLOCKS = ROWB >= 256 ? 2 : (ROWS == 8 ? 4 : 3);
  static constexpr int META = NW * STAGES * 16;
  static constexpr int QS = E4M3 ? 1 : 2;   // terms of Q
  static constexpr int SMEM = RING + META + QS * ROWS * QP * 2 + ROWS * 4 + 2 * NW * ROWS * 4;
  static_assert((NW + 1) * ROWS * D * 4 <= RING, "the warps' O and their sum must fit the ring");
};

// All threads of all blocks of the cluster; orders their shared memory accesses.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same place in the shared memory of block `rank` of the cluster.
template <class T>
__device__ __forceinline__ const T* cluster_ptr(const T* p, int rank) {
  uint64_t q;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<const T*>(q);
}

// Four elements of a finished row: O / L (a row that saw no key: 0), and its lse.
__device__ __forceinline__ void store_row(const PagedAttnParams& p, size_t at, int d4, int D, const float4& a, float M,
                                          float L) {
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(p.out + at * D + d4 * 4) =
      make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (p.lse != nullptr && d4 == 0) p.lse[at] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int CH>
__device__ __forceinline__ int swz(int row, int c) {
  if constexpr (CH == 4) return c ^ ((row >> 1) & 3);
  return c ^ ((((row ^ (row >> 2)) & 1) << 2) | (row & 2));
}

template <class TR, int MODS>
__global__ void __launch_bounds__(TR::THREADS, TR::BLOCKS) paged_decode_kernel(const PagedAttnParams p) {
  constexpr int D = TR::D, CH = TR::CH, NW = TR::NW, STAGES = TR::STAGES, TILE = TR::TILE;
  constexpr int ROWS = TR::ROWS, NR = TR::NR, MT = TR::MT;
  constexpr bool E4M3 = TR::E4M3;
  constexpr float HEAD = kHeadroom<E4M3>, UNIT = 1.f / (1 << kSumUnit<E4M3>);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* s_ring = smem;
  float* s_meta = reinterpret_cast<float*>(smem + TR::RING);  // [NW][STAGES][4]: K scale, V scale, page mapped
  uint16_t* s_q = reinterpret_cast<uint16_t*>(smem + TR::RING + TR::META);  // [QS][ROWS][QP]
  float* s_qf = reinterpret_cast<float*>(s_q + TR::QS * ROWS * TR::QP);     // [ROWS]
  float* s_m = s_qf + ROWS;                                                 // [NW][ROWS]
  float* s_l = s_m + NW * ROWS;

  asm volatile("griddepcontrol.launch_dependents;");
  const int split = blockIdx.x % p.nsplit, rt = blockIdx.x / p.nsplit;
  const int hkv = blockIdx.y, b = blockIdx.z;
  const int ps = p.pool.page_size;
  const SeqView s = seq_view(p.batch, b);
  const int rows = s.nq * p.group, r0 = rt * ROWS;
  if (r0 >= rows) return;  // all blocks of the cluster
  int p_lo, p_hi;
  unit_positions(p, s, r0, p_lo, p_hi);
  const KeyRange kr = key_range(p.sc, b, s, p_lo, p_hi, 16);
  const int pieces = p.clustered ? p.nsplit : piece_count(p, kr.nt);
  if (split >= pieces) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster shares its unit's keys evenly
  const int even = (kr.nt + pieces - 1) / pieces;
  const int t_beg = (p.clustered ? split * even : piece_begin(p, split)) + warp;
  const int t_end = p.clustered ? min(kr.nt, (split + 1) * even) : piece_end(p, split, pieces, kr.nt);
  const int n_my = t_end > t_beg ? (t_end - t_beg + NW - 1) / NW : 0;

  // ---- the ring
  const uint32_t ring = smem_addr(s_ring) + warp * (STAGES * 2 * TILE);
  const uint32_t meta = smem_addr(s_meta) + warp * (STAGES * 16);
  int my_page = -1;
  auto issue = [&](int k) {
    if (k < n_my) {
      if ((k & 31) == 0) {  // the pages of this warp's next 32 tiles, one per lane
        const int kk = k + lane;
        my_page = kk < n_my ? page_of(p.batch, b, kr.tile(t_beg + kk * NW) * 16 >> p.pool.page_shift, p.pool.n_pages) : -1;
      }
      const int page = __shfl_sync(0xffffffffu, my_page, k & 31);
      const int key0 = kr.tile(t_beg + k * NW) * 16;
      const int st = k % STAGES;
      const size_t head = static_cast<size_t>(page < 0 ? 0 : page) * p.pool.H + hkv;
      const size_t src = (head * ps + (key0 & (ps - 1))) * TR::ROWB + lane * 16;
      const uint8_t* kfrom = static_cast<const uint8_t*>(p.pool.k) + src;
      const uint8_t* vfrom = static_cast<const uint8_t*>(p.pool.v) + src;
      const uint32_t dst = ring + st * (2 * TILE);
      // every key is seen by some row, or each is looked at
      const bool whole = key0 + 16 <= kr.always || (key0 >= kr.lo && key0 + 16 <= kr.upper);
      auto copy = [&](auto all) {
#pragma unroll
        for (int i = 0; i < TILE / 512; ++i) {
          const int c = lane + 32 * i, row = c / CH, ch = c % CH;
          const bool ok = page >= 0 && (all || kr.some_row_sees(key0 + row));
          const uint32_t to = dst + row * TR::ROWB + (swz<CH>(row, ch) << 4);
          cp_async16(to, kfrom + i * 512, ok);
          cp_async16(to + TILE, vfrom + i * 512, ok);
        }
      };
      if (whole) copy(std::true_type{});
      else copy(std::false_type{});
      if constexpr (E4M3) {
        if (lane < 2) cp_async4(meta + st * 16 + lane * 4, (lane ? p.pool.v_scale : p.pool.k_scale) + head, page >= 0);
      }
      if (lane == 2) s_meta[(warp * STAGES + st) * 4 + 2] = page >= 0 ? 1.f : 0.f;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) issue(k);

  // ---- Q: rotated in fp32, rounded to the MMA's type
  __shared__ unsigned long long s_turns[kMaxTokenPairs];
  if (p.rope.rot > 0) {
    if (threadIdx.x < p.rope.rot >> 1) s_turns[threadIdx.x] = p.rope.turns[threadIdx.x];
    __syncthreads();
  }
  for (int i = threadIdx.x; i < ROWS * (D / 16); i += TR::THREADS) {
    const int r = i / (D / 16), c = i % (D / 16);
    const int row = r0 + r, tok = row / p.group, h = hkv * p.group + row % p.group;
    int lo, hi;
    item_chunks(p.rope, c, lo, hi);
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
    if (row < rows) {
      const __nv_bfloat16* src = p.q + (s.q0 + tok) * p.q_stride + h * D;
      load_chunk8<__nv_bfloat16>(src + lo * 8, x);
      load_chunk8<__nv_bfloat16>(src + hi * 8, y);
      if (c < (p.rope.rot >> 4)) {
        float2 cs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = turn_of(p.rope, s.first_pos + tok, s_turns[c * 8 + e]);
        rotate_item(p.rope, x, y, cs, 1);
      }
    }
    uint32_t w[8];
    if constexpr (E4M3) {
      // fp16 has bf16's precision and three bits more, but a short range: the
      // row is divided by the power of two below its largest element
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmax3(a, fabsf(x[e]), fabsf(y[e]));
#pragma unroll
      for (int o = D / 32; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float f = power_below(a), inv = 1.f / f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = pack_f16(x[2 * e] * inv, x[2 * e + 1] * inv);
        w[4 + e] = pack_f16(y[2 * e] * inv, y[2 * e + 1] * inv);
      }
      if (c == 0) s_qf[r] = f;
    } else {
      // two bf16 terms: a rotated q keeps 16 bits, for MMAs that the loads hide (one
      // term: error 3.5e-3 of the output, two: 2.2e-3, of which 1.7e-3 is its rounding)
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = e < 4 ? x[2 * (e & 3)] : y[2 * (e & 3)], b2 = e < 4 ? x[2 * (e & 3) + 1] : y[2 * (e & 3) + 1];
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b2);
        const float2 f2 = __bfloat1622float2(h2);
        w[e] = *reinterpret_cast<const uint32_t*>(&h2);
        v[e] = pack_bf16(a - f2.x, b2 - f2.y);
      }
      uint16_t* s_lo = s_q + ROWS * TR::QP + r * TR::QP;
      *reinterpret_cast<uint4*>(s_lo + lo * 8) = make_uint4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<uint4*>(s_lo + hi * 8) = make_uint4(v[4], v[5], v[6], v[7]);
      if (c == 0) s_qf[r] = 1.f;
    }
    *reinterpret_cast<uint4*>(s_q + r * TR::QP + lo * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(s_q + r * TR::QP + hi * 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __syncthreads();

  const int g = lane >> 2, t = lane & 3;
  uint32_t bq[NR][TR::KS][2];
  // this lane's query rows: 2t + q + 8r at [2r + q]
  float fac[2 * NR], slope[2 * NR];
  int pos[2 * NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int j = 0; j < TR::KS; ++j) {
      constexpr int U = TR::EPC / 4;  // MMAs per chunk
      const int d = (t + 4 * (j / U)) * TR::EPC + 4 * (j % U);
      const uint2 u = *reinterpret_cast<const uint2*>(s_q + (g + 8 * r) * TR::QP + d);
      bq[r][j][0] = u.x;
      bq[r][j][1] = u.y;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = 2 * t + q + 8 * r;
      fac[2 * r + q] = s_qf[row] * p.sc.pre;
      pos[2 * r + q] = s.first_pos + (r0 + row) / p.group;
      slope[2 * r + q] = MODS & kBiased ? p.sc.slope2[hkv * p.group + (r0 + row) % p.group] : 0.f;
    }
  }

  float o[NR][MT][4];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][n][e] = 0.f;
  // m: reference of the row's exponents (a running max less the headroom, raised only when
  // it is exceeded by 2^8: sums and O are rescaled rarely); l: this lane's share of the
  // sum. Over an 8-bit pool V's codes enter the MMA as they are and their scale
  // goes with P = p vs, so the reference is the max of x + c, c the scale's exponent: P then
  // stays inside fp16 whatever the pages' scales are.
  float m[2 * NR], l[2 * NR];
#pragma unroll
  for (int q = 0; q < 2 * NR; ++q) m[q] = -INFINITY, l[q] = 0.f;

  for (int k = 0; k < n_my; ++k) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    const int st = k % STAGES;
    const uint8_t* sk = s_ring + warp * (STAGES * 2 * TILE) + st * (2 * TILE);
    const uint8_t* sv = sk + TILE;
    const float4 mt = *reinterpret_cast<const float4*>(s_meta + (warp * STAGES + st) * 4);
    const int key0 = kr.tile(t_beg + k * NW) * 16;
    // S^T: [key g: row 2t, 2t+1][key g + 8: row 2t, 2t+1]
    // (two accumulators, so that the MMAs' latencies overlap)
    float sx[NR][4], sy[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) sx[r][e] = sy[r][e] = 0.f;
#pragma unroll
    for (int i = 0; i < TR::KC; ++i) {
      const int ch = swz<CH>(g, t + 4 * i) << 4;  // g + 8 is swizzled like g
      const uint4 u = *reinterpret_cast<const uint4*>(sk + g * TR::ROWB + ch);
      const uint4 w = *reinterpret_cast<const uint4*>(sk + (g + 8) * TR::ROWB + ch);
      const uint32_t ua[4] = {u.x, u.y, u.z, u.w}, wa[4] = {w.x, w.y, w.z, w.w};
      if constexpr (E4M3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_f16(ua[e], a0, a2);
          e4m3x4_f16(wa[e], a1, a3);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            mma16816<true>(e & 1 ? sy[r] : sx[r], a0, a1, a2, a3, bq[r][i * 4 + e][0], bq[r][i * 4 + e][1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int r = 0; r < NR; ++r)
            mma16816<false>(e & 1 ? sy[r] : sx[r], ua[2 * e], wa[2 * e], ua[2 * e + 1], wa[2 * e + 1],
                            bq[r][i * 2 + e][0], bq[r][i * 2 + e][1]);
        if (p.rope.rot > 0) {  // an unrotated q is bf16 as it stands
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const uint2 q2 = *reinterpret_cast<const uint2*>(s_q + (ROWS + g + 8 * r) * TR::QP + (t + 4 * i) * 8 + 4 * e);
              mma16816<false>(e & 1 ? sx[r] : sy[r], ua[2 * e], wa[2 * e], ua[2 * e + 1], wa[2 * e + 1], q2.x, q2.y);
            }
        }
      }
    }
    // scores in log2 units
    const float ks = E4M3 ? mt.x : 1.f;
    with_cap<MODS>(p.sc, [&](auto wide) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = fac[2 * r + (e & 1)] * ks, y = sx[r][e] + sy[r][e];
          const int q = 2 * r + (e & 1);
          sx[r][e] = score2<MODS, decltype(wide)::value>(p.sc, y, f, slope[q],
                                                         MODS & kBiased ? offset_of(pos[q], key0 + g + 8 * (e >> 1)) : 0.f);
        }
    });
    const bool all_seen = mt.z != 0.f && (key0 + 16 <= kr.prefix ||
                                          (key0 + 15 <= p_lo && key0 + 16 <= s.len &&
                                           (p.sc.window == 0 || p_hi - key0 < p.sc.window)));
    if (!all_seen) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = key0 + g + 8 * (e >> 1);
          if (mt.z == 0.f || !row_sees(p.sc, kr, s.len, pos[2 * r + (e & 1)], j)) sx[r][e] = -INFINITY;
        }
    }
    const int ce = E4M3 ? scale_exponent(mt.y) : 0;
    const float c2 = static_cast<float>(ce);
    const float inv_c = E4M3 ? power_of_two(-ce) : 1.f, mant = E4M3 ? mt.y * inv_c : 1.f;
    const float share = inv_c * UNIT;  // of P, in the sum
    bool raise = false;
#pragma unroll
    for (int q = 0; q < 2 * NR; ++q)
      raise = raise || fmaxf(sx[q >> 1][q & 1], sx[q >> 1][2 + (q & 1)]) + c2 > m[q] + (8.f + HEAD);
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int q = 0; q < 2 * NR; ++q) {
        float mx = fmaxf(sx[q >> 1][q & 1], sx[q >> 1][2 + (q & 1)]) + c2;
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float nm = fmaxf(m[q], mx - HEAD);
        const float al = nm == -INFINITY ? 1.f : ex2(m[q] - nm);
        m[q] = nm;
        l[q] *= al;
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          o[q >> 1][n][q & 1] *= al;
          o[q >> 1][n][2 + (q & 1)] *= al;
        }
      }
    }
    uint32_t pb[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float m0 = m[2 * r] == -INFINITY ? 0.f : m[2 * r], m1 = m[2 * r + 1] == -INFINITY ? 0.f : m[2 * r + 1];
      const float f0 = c2 - m0, f1 = c2 - m1;
      const float e0 = ex2(sx[r][0] + f0), e1 = ex2(sx[r][1] + f1), e2 = ex2(sx[r][2] + f0), e3 = ex2(sx[r][3] + f1);
      l[2 * r] = fmaf(e0 + e2, share, l[2 * r]);
      l[2 * r + 1] = fmaf(e1 + e3, share, l[2 * r + 1]);
      if constexpr (E4M3) {
        pb[r][0] = transpose8x8(pack_f16(e0 * mant, e1 * mant));
        pb[r][1] = transpose8x8(pack_f16(e2 * mant, e3 * mant));
      } else {
        pb[r][0] = transpose8x8(pack_bf16(e0, e1));
        pb[r][1] = transpose8x8(pack_bf16(e2, e3));
      }
    }
    // O^T += V^T P^T; words w[q] of key 2t, 2t+1, 2t+8, 2t+9
    auto pv = [&](int n, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int r = 0; r < NR; ++r) mma16816<E4M3>(o[r][n], a0, a1, a2, a3, pb[r][0], pb[r][1]);
    };
    auto pv_word = [&](int n, const uint32_t (&w)[4]) {
      if constexpr (E4M3) {  // four d: two MMAs
        uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
        e4m3x4_f16(__byte_perm(w[0], w[1], 0x5140), x0, x1);
        e4m3x4_f16(__byte_perm(w[0], w[1], 0x7362), x2, x3);
        e4m3x4_f16(__byte_perm(w[2], w[3], 0x5140), y0, y1);
        e4m3x4_f16(__byte_perm(w[2], w[3], 0x7362), y2, y3);
        pv(2 * n, x0, x1, y0, y1);
        pv(2 * n + 1, x2, x3, y2, y3);
      } else {  // two d: one MMA
        pv(n, __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x5410),
           __byte_perm(w[2], w[3], 0x7632));
      }
    };
    if constexpr (CH == 4) {  // 64-byte rows: half a chunk per lane
      uint2 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 2 * t + (q & 1) + 8 * (q >> 1);
        u[q] = *reinterpret_cast<const uint2*>(sv + row * TR::ROWB + (swz<CH>(row, g >> 1) << 4) + (g & 1) * 8);
      }
      pv_word(0, {u[0].x, u[1].x, u[2].x, u[3].x});
      pv_word(1, {u[0].y, u[1].y, u[2].y, u[3].y});
    } else {
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) {
        uint4 u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = 2 * t + (q & 1) + 8 * (q >> 1);
          u[q] = *reinterpret_cast<const uint4*>(sv + row * TR::ROWB + (swz<CH>(row, g + 8 * i) << 4));
        }
        pv_word(4 * i, {u[0].x, u[1].x, u[2].x, u[3].x});
        pv_word(4 * i + 1, {u[0].y, u[1].y, u[2].y, u[3].y});
        pv_word(4 * i + 2, {u[0].z, u[1].z, u[2].z, u[3].z});
        pv_word(4 * i + 3, {u[0].w, u[1].w, u[2].w, u[3].w});
      }
    }
    __syncwarp();  // every lane is done with the stage
    issue(k + STAGES - 1);
  }

  // ---- join the block's warps
  // (sums and O in the same units from here on)
  cp_async_wait<0>();
#pragma unroll
  for (int q = 0; q < 2 * NR; ++q) m[q] += static_cast<float>(kSumUnit<E4M3>);
#pragma unroll
  for (int q = 0; q < 2 * NR; ++q)
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) l[q] += __shfl_xor_sync(0xffffffffu, l[q], w);
  if (g == 0)
#pragma unroll
    for (int q = 0; q < 2 * NR; ++q) {
      s_m[warp * ROWS + 2 * t + (q & 1) + 8 * (q >> 1)] = m[q];
      s_l[warp * ROWS + 2 * t + (q & 1) + 8 * (q >> 1)] = l[q];
    }
  __syncthreads();
  float* s_o = reinterpret_cast<float*>(s_ring);  // [NW][ROWS][D]
  float* c_o = s_o + NW * ROWS * D;               // [ROWS][D]: the block's sum, for its cluster
  float2* c_ml = reinterpret_cast<float2*>(s_q);  // [ROWS]: Q is done with
#pragma unroll
  for (int q = 0; q < 2 * NR; ++q) {
    const int row = 2 * t + (q & 1) + 8 * (q >> 1);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * ROWS + row]);
    const float f = m[q] == -INFINITY ? 0.f : ex2(m[q] - M) * UNIT;
    float* dst = s_o + (warp * ROWS + row) * D;
#pragma unroll
    for (int n = 0; n < MT; ++n) {
      // the two d of MMA n in lane g
      const int d = E4M3 ? g * (D / 8) + 2 * n : (g + 8 * (n / 4)) * 8 + 2 * (n % 4);
      *reinterpret_cast<float2*>(dst + d) = make_float2(o[q >> 1][n][q & 1] * f, o[q >> 1][n][2 + (q & 1)] * f);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += TR::THREADS) {
    const int r = i / (D / 4), d4 = i % (D / 4);
    const int row = r0 + r;
    if (row >= rows) break;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * ROWS + r]);
#pragma unroll
    for (int w = 0; w < NW; ++w) L += M == -INFINITY ? 0.f : s_l[w * ROWS + r] * ex2(s_m[w * ROWS + r] - M);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(s_o + (w * ROWS + r) * D + d4 * 4);
      a.x += u.x;
      a.y += u.y;
      a.z += u.z;
      a.w += u.w;
    }
    const size_t at = static_cast<size_t>(s.q0 + row / p.group) * p.Hq + hkv * p.group + row % p.group;
    if (pieces == 1) {
      store_row(p, at, d4, D, a, M, L);
    } else if (p.clustered) {
      *reinterpret_cast<float4*>(c_o + r * D + d4 * 4) = a;
      if (d4 == 0) c_ml[r] = make_float2(M, L);
    } else {
      __stcg(reinterpret_cast<float4*>(p.part_o + (at * p.nsplit + split) * D + d4 * 4), a);
      if (d4 == 0) __stcg(p.part_ml + at * p.nsplit + split, make_float2(M, L));
    }
  }
  if (p.clustered && pieces > 1) {
    // the cluster's blocks join their rows through each other's shared memory, a share
    // of the elements each
    __syncwarp();
    cluster_barrier();
    for (int i = threadIdx.x + split * TR::THREADS; i < ROWS * (D / 4); i += pieces * TR::THREADS) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      const int row = r0 + r;
      if (row >= rows) break;
      float M = -INFINITY, L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < pieces; ++c) {
        const float2 ml = *reinterpret_cast<const float2*>(cluster_ptr(c_ml + r, c));
        const float4 u = *reinterpret_cast<const float4*>(cluster_ptr(c_o + r * D + d4 * 4, c));
        const float nm = fmaxf(M, ml.x);
        const float f0 = M == -INFINITY ? 0.f : ex2(M - nm), f1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - nm);
        M = nm;
        L = L * f0 + ml.y * f1;
        a.x = a.x * f0 + u.x * f1;
        a.y = a.y * f0 + u.y * f1;
        a.z = a.z * f0 + u.z * f1;
        a.w = a.w * f0 + u.w * f1;
      }
      const size_t at = static_cast<size_t>(s.q0 + row / p.group) * p.Hq + hkv * p.group + row % p.group;
      store_row(p, at, d4, D, a, M, L);
    }
    __syncwarp();
    cluster_barrier();  // nobody leaves while its shared memory is read
  }
}

// ---------------------------------------------------------------------------
// Joins the pieces of every row whose key range was split: one block per (row, query
// head), its warps taking pieces in turn. Launched behind the kernel that wrote them,
// whose end it awaits on the device (programmatic dependent launch).
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedAttnParams p) {
  constexpr int NW = kJoinThreads / 32, V = D / 32;  // elements per lane
  __shared__ float2 s_ml[NW];
  __shared__ float s_o[NW][D];
  const int b = blockIdx.y;
  const SeqView s = seq_view(p.batch, b);
  const int tok = blockIdx.x / p.Hq, h = blockIdx.x - tok * p.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int pieces = 1;
  if (tok < s.nq) {
    const int row = tok * p.group + h % p.group;
    int lo, hi;
    unit_positions(p, s, row / p.row_tile * p.row_tile, lo, hi);
    pieces = piece_count(p, key_range(p.sc, b, s, lo, hi, p.key_tile).nt);
  }
  // every thread waits, those without work too: this kernel's end has to stand for the pieces' kernel's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (pieces == 1) return;
  const size_t at = static_cast<size_t>(s.q0 + tok) * p.Hq + h;
  const float2* ml = p.part_ml + at * p.nsplit;
  const float* src = p.part_o + at * p.nsplit * D + lane * V;
  float M = -INFINITY, L = 0.f, a[V];
#pragma unroll
  for (int e = 0; e < V; ++e) a[e] = 0.f;
  constexpr int U = 4;  // pieces in flight per warp
  for (int i0 = warp; i0 < pieces; i0 += NW * U) {
    float2 u[U];
    float v[U][V];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * NW < pieces ? i0 + k * NW : i0;
      u[k] = __ldcg(ml + i);
      if (i0 + k * NW >= pieces) u[k].x = -INFINITY;
      if constexpr (V == 4) {
        const float4 q = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(i) * D));
        v[k][0] = q.x; v[k][1] = q.y; v[k][2] = q.z; v[k][3] = q.w;
      } else {
        const float2 q = __ldcg(reinterpret_cast<const float2*>(src + static_cast<size_t>(i) * D));
        v[k][0] = q.x; v[k][1] = q.y;
      }
    }
    float nm = M;
#pragma unroll
    for (int k = 0; k < U; ++k) nm = fmaxf(nm, u[k].x);
    if (nm == -INFINITY) continue;
    const float f = ex2(M - nm);
    M = nm;
    L *= f;
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] *= f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float g = ex2(u[k].x - nm);
      L += u[k].y * g;
#pragma unroll
      for (int e = 0; e < V; ++e) a[e] += v[k][e] * g;
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = a[e];
  if (lane == 0) s_ml[warp] = make_float2(M, L);
  __syncthreads();
  const int d4 = threadIdx.x;
  if (d4 >= D / 4) return;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w].x);
  L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(s_ml[w].x - M);
      const float4 q = *reinterpret_cast<const float4*>(&s_o[w][d4 * 4]);
      L += s_ml[w].y * f;
      o.x += q.x * f;
      o.y += q.y * f;
      o.z += q.z * f;
      o.w += q.w * f;
    }
  store_row(p, at, d4, D, o, M, L);
}

}  // namespace ll
