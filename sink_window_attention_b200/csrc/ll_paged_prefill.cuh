// ll_paged_prefill.cuh — attention of many rows (prompts, chunks) over a paged
// pool on the tcgen05 tensor cores.
//
// One CTA: up to 256 rows (token, query head of the group) of a sequence and K/V
// head as two tiles of 128, against a piece of its keys in tiles of 128.
//  * warps 0-3 gather K and V tiles out of the pages into a ring of shared-memory
//    buffers in the 128-byte-swizzled operand layout, K_0 V_0 K_1 V_1 ...: a BF16
//    pool by cp.async, an 8-bit one through registers, where E4M3 becomes fp16
//    (exact). Plain loads rather than TMA boxes because a key tile is 1 to 8
//    pages, rows that nobody sees are left out (read as zeros) row by row, and the
//    8-bit tile has to pass through registers anyhow.
//  * warp 4 issues the MMAs: S_w = Q_w K_i^T (both operands in shared memory) and
//    O_w += P_w V_i (P in tensor memory, over S_w's columns), for the row tiles
//    w = A, B in turn: one tile's softmax runs under the other's MMAs, which also keeps
//    the two from wanting the exponential unit at the same time. P is handed over in
//    halves, so P V begins under the second half's exponentials. (S in halves of 64
//    keys, double-buffered, so that no softmax ever waited for its own MMAs, ran both
//    softmaxes in lockstep and was slower: 599 us against 565 then.)
//  * warps 8-11 and 12-15 are A's and B's softmax, a row per thread: maxima and
//    sums in fp32; O is rescaled in tensor memory only when the reference is
//    exceeded by 2^8 (2^14 over an 8-bit pool, where it starts 2^6 below the maximum).
// 1024 queries of 32 heads over 32768 keys (8 K/V heads of 128): 528 us alone, 1020 TFLOP/s,
// over a bf16 pool (599 replayed 20 times in a row, at the power limit), 612 (621) us over
// an 8-bit one (its softmax reads the groups' scales, spills some 80 bytes a thread and has
// 4 operand buffers instead of 5). Per 256 x 128 tile of the latter 4700 clocks (1.067 million of the kernel over 227 tiles): tensor pipe 45 % active,
// exponential unit 46 %, issue slots 47 %. What neither covers is one softmax warp per row
// tile and scheduler waiting for its own results; it is not located further. A CTA takes
// about 6 us to start (lengths, pages, Q, first tiles) and end.
// 8-bit pools: a group of 16 keys lies in one page, so its K scale is a factor and
// the exponent of its V scale an offset per 16 scores; the V scale's mantissa (1
// for the powers of two that the append writes) is multiplied into V's fp16.
#pragma once

#include <type_traits>

#include "ll_paged_attention.cuh"

namespace ll {

template <int D_, bool E4M3_>
struct PrefillTraits {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int BM = 128, BN = 128, HN = 64;  // rows, keys of a tile, keys of a half
  static constexpr int NB = D / 64;              // 128-byte column blocks of a row
  static constexpr int TILE = BN * D * 2;        // one K, V or Q operand tile
  static constexpr int CTRL = 2048;
  // 8-bit pools: a tile's codes of K and V on their way to fp16
  static constexpr int RAW = E4M3 ? 2 * BN * D : 0;
  // Terms of a rotated q. One bf16 term rounds each element by up to 2^-8 (output error
  // 3.6e-3 of its norm, with two terms 2.3e-3). At D = 64 two more tiles of 16 KB fit beside
  // the buffers and the second product hides (ragged prompts of 32 heads: 218 us rotated, 202
  // not). At D = 128 they would leave 3 of 5 buffers, and the products would be most of a
  // tile's time: ragged prompts 249 -> 285 us, a chunk of 1024 over 32768 582 -> 711, so
  // there one term stays. fp16 (8-bit pools) has three bits more in one.
  static constexpr int QS = !E4M3 && D == 64 ? 2 : 1;
  static constexpr int FREE = (232448 - CTRL - 1024 - RAW) / TILE - 2 * QS;
  static constexpr int STAGES = FREE < 8 ? FREE : 8;
  static constexpr int SMEM = CTRL + 1024 + (2 * QS + STAGES) * TILE + RAW;
  // Slots of per-tile page data. Slot i is written again with buffer K_(i+META),
  // which can only be filled once V_i was consumed (2 META - STAGES >= 1), that is
  // after both softmax warpgroups handed over P_i and so have read slot i.
  static constexpr int META = STAGES / 2 + 1;
  static_assert(2 * META - STAGES >= 1, "meta slots");
  static constexpr int THREADS = 512;
  // registers: launch 128 per thread (512 x 128 = 65536); loaders 80, the MMA
  // issuer's warpgroup 48, the softmax warpgroups 192: 80 + 48 + 2 x 192 = 4 x 128
  static constexpr int LAUNCH_REGS = 128, REGS_LOAD = 80, REGS_MMA = 48, REGS_SOFTMAX = 192;
  static_assert(REGS_LOAD + REGS_MMA + 2 * REGS_SOFTMAX <= 4 * LAUNCH_REGS, "register split exceeds the launch");
  static constexpr int TMEM_COLS = 512, S_COL = 0, O_COL = 2 * BN;
  static constexpr int FMT = E4M3 ? 0 : 1;       // kind::f16 operands: f16 or bf16
  static_assert(STAGES >= (E4M3 ? 4 : 5), "buffers that the issue order needs: K, V of a tile, the next K, and those in flight");
};

// What the softmax has to know of 16 keys that lie in one page.
struct KeyGroup {
  float ks;      // K scale
  float c;       // exponent of the V scale
  float share;   // 2^-c in units of the sum
  float unused;
};

// What two values lose when they are rounded to bf16, as bf16.
__device__ __forceinline__ uint32_t pack_bf16_rest(float a, float b) {
  const float2 f = __bfloat1622float2(__floats2bfloat162_rn(a, b));
  return pack_bf16(a - f.x, b - f.y);
}

// Like turn_of, with the hardware's sine and cosine of at most an eighth of a
// turn (within 2^-21): for queries, which keep 11 to 16 bits right after.
__device__ __forceinline__ float2 turn_fast(const TokenRope& r, int pos, int i) {
  const uint32_t t = turned(pos, r.turns[i]);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int>(t - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  float s, c;
  __sincosf(a, &s, &c);
  float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  if ((quarter + 1) & 2) x = -x;
  if (quarter & 2) y = -y;
  return make_float2(x * r.amp, y * r.amp);
}

// mbar_wait for the loaders, who are buffers ahead: they sleep between polls, which
// would take issue slots from the softmax.
__device__ __forceinline__ bool mbar_wait_sleeping(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_addr(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(&g_error_word, kErrWaitTimeout);
      *abort = 1;
      return false;
    }
    __nanosleep(100);
  }
  return true;
}

template <class TR, int MODS>
__global__ void __launch_bounds__(TR::THREADS, 1) paged_prefill_kernel(const PagedAttnParams p) {
  constexpr int D = TR::D, BM = TR::BM, BN = TR::BN, STAGES = TR::STAGES, TILE = TR::TILE;
  constexpr bool E4M3 = TR::E4M3;
  constexpr float HEAD = kHeadroom<E4M3>, UNIT = 1.f / (1 << kSumUnit<E4M3>);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                      // [2][QS][TILE]
  uint8_t* sKV = smem + 2 * TR::QS * TILE;  // [STAGES][TILE]
  uint8_t* sRaw = sKV + STAGES * TILE;  // [2][BN / RPS][128] chunks
  uint8_t* ctrl = sRaw + TR::RAW;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);  // [STAGES]
  uint64_t* empty = full + 8;                          // [STAGES]
  uint64_t* meta_full = empty + 8;                     // [META]
  uint64_t* q_full = meta_full + TR::META;
  uint64_t* s_full = q_full + 1;   // [2] row tile
  uint64_t* p_ready = s_full + 2;  // [2][2] row tile, half of the keys
  uint64_t* o_done = p_ready + 4;  // [2]
  uint64_t* drain = o_done + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* meta_mapped = const_cast<int*>(s_abort) + 1;           // [META]: bit g: keys [16 g, 16 g + 16) have a page
  KeyGroup* meta = reinterpret_cast<KeyGroup*>(ctrl + 512);  // [META][8]
  static_assert((8 + 8 + TR::META + 10) * 8 + 8 + TR::META * 4 <= 512 && 512 + TR::META * 8 * sizeof(KeyGroup) <= TR::CTRL, "control block");

  asm volatile("griddepcontrol.launch_dependents;");
  // the last rows of a sequence see the most keys: those of all sequences start first
  // (and a range's first piece, which may be the longer, before the others)
  const int hkv = blockIdx.x, b = blockIdx.y;
  const int split = blockIdx.z / p.row_tiles, rt = p.row_tiles - 1 - blockIdx.z % p.row_tiles;
  const int ps = p.pool.page_size;
  const SeqView s = seq_view(p.batch, b);
  const int rows = s.nq * p.group, r0 = rt * 2 * BM;
  if (r0 >= rows) return;
  int p_lo, p_hi;
  unit_positions(p, s, r0, p_lo, p_hi);
  const KeyRange kr = key_range(p.sc, b, s, p_lo, p_hi, BN);
  const int pieces = piece_count(p, kr.nt);
  if (split >= pieces) return;
  const int t_beg = piece_begin(p, split);
  const int n = piece_end(p, split, pieces, kr.nt) - t_beg;  // key tiles of this piece (0: nothing is seen)
  const bool two = rows - r0 > BM;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 128);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < TR::META; ++i) mbar_init(&meta_full[i], 1);
    mbar_init(q_full, two ? 256 : 128);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_ready[2 * w], 128);
      mbar_init(&p_ready[2 * w + 1], 128);
      mbar_init(&o_done[w], 1);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(s_tmem, TR::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *s_tmem;

  if (warp < 4) {
    // ------------------------------------------------------------ loaders
    regs_dec<TR::REGS_LOAD>();
    const int tid = threadIdx.x;
    // Lane g < 8 holds the place of keys [16 g, 16 g + 16) of a tile, which lie in
    // one page: their page (-1: none, or no row sees one of them: neither their rows nor
    // their scales are read then) and their number in the pool's runs of 16 rows.
    const int per_page = ps >> 4;
    auto page_for = [&](int i) -> int {
      if (lane >= 8 || i >= n) return -1;
      const int key = kr.tile(t_beg + i) * BN + lane * 16;
      const bool seen = key < kr.always || (key + 16 > kr.lo && key < kr.upper);
      return seen ? page_of(p.batch, b, key >> p.pool.page_shift, p.pool.n_pages) : -1;
    };
    auto run_of = [&](int i, int page) -> int {
      return page < 0 ? -1 : (page * p.pool.H + hkv) * per_page + ((kr.tile(t_beg + i) * 8 + lane) & (per_page - 1));
    };
    auto scale_for = [&](const float* scales, int page) -> float {
      return E4M3 && page >= 0 ? scales[static_cast<size_t>(page) * p.pool.H + hkv] : 0.f;
    };
    int pg = page_for(0), pg1 = page_for(1);
    float ks = scale_for(p.pool.k_scale, pg), vs = scale_for(p.pool.v_scale, pg);
    bool ok = true;
    // this thread's writes of buffer `pos` are done
    auto publish = [&](int st) {
      fence_proxy_async_smem();
      mbar_arrive(&full[st]);
    };
    auto wait_empty = [&](int st, int round) {
      if (ok) ok = mbar_wait_sleeping(&empty[st], (round & 1) ^ 1, s_abort);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto put_meta = [&](int i) {
      if (warp == 0) {
        const unsigned mapped = __ballot_sync(0xffffffffu, pg >= 0);
        if (lane == 0) meta_mapped[i % TR::META] = static_cast<int>(mapped);
        if (E4M3 && lane < 8) {
          const int c = scale_exponent(vs);
          meta[(i % TR::META) * 8 + lane] = KeyGroup{ks, static_cast<float>(c), power_of_two(-c) * UNIT, 0.f};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&meta_full[i % TR::META]);
      }
    };
    // every row of a tile is seen by some row of the unit: nothing to leave out
    auto whole_tile = [&](int key0) { return key0 + BN <= kr.always || (key0 >= kr.lo && key0 + BN <= kr.upper); };
    int st = 0, round = 0;  // buffer and its use
    if constexpr (!E4M3) {
      constexpr int CPR = D / 8, RPS = 128 / CPR, PER_RUN = 16 / RPS;  // chunks per row, rows per step, steps per run
      constexpr int AHEAD = 2;  // buffers in flight behind the one being issued
      const int c = tid % CPR, r = tid / CPR;
      const uint32_t dst0 = smem_addr(sKV) + (c >> 3) * (BN * 128) + sw128_offset(r, c & 7);
      const size_t lane_off = static_cast<size_t>(r) * (D * 2) + c * 16;
      int behind = 0, behind_st = 0;  // buffers issued but not published, and the oldest of them
      for (int i = 0; i < n && ok; ++i) {
        const int pg2 = page_for(i + 2);
        const int key0 = kr.tile(t_beg + i) * BN;
        const int run = run_of(i, pg);
        const bool whole = whole_tile(key0);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          wait_empty(st, round);
          if (!ok) break;
          const uint8_t* src = static_cast<const uint8_t*>(kv ? p.pool.v : p.pool.k) + lane_off;
          const uint32_t dst = dst0 + st * TILE;
          // a run's rows are whole 8-row swizzle atoms apart, so the swizzle is r's
          auto copy = [&](auto all) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const int at = __shfl_sync(0xffffffffu, run, g);
              const uint8_t* from = src + static_cast<size_t>(at < 0 ? 0 : at) * (16 * D * 2);
#pragma unroll
              for (int k = 0; k < PER_RUN; ++k) {
                const int row = g * 16 + k * RPS;  // + r
                const bool valid = at >= 0 && (all || kr.some_row_sees(key0 + row + r));
                cp_async16(dst + row * 128, from + k * (RPS * D * 2), valid);
              }
            }
          };
          if (whole) copy(std::true_type{});
          else copy(std::false_type{});
          cp_async_commit();
          if (kv == 0) put_meta(i);
          if (++behind > AHEAD) {
            cp_async_wait<AHEAD>();
            publish(behind_st);
            --behind;
            if (++behind_st == STAGES) behind_st = 0;
          }
          if (++st == STAGES) st = 0, ++round;
        }
        pg = pg1;
        pg1 = pg2;
      }
      cp_async_wait<0>();
      if (ok)
        for (; behind > 0; --behind) {
          publish(behind_st);
          if (++behind_st == STAGES) behind_st = 0;
        }
    } else {
      constexpr int CPR = D / 16, RPS = 128 / CPR, STEPS = BN / RPS;  // 16-code chunks per row
      const int c = tid % CPR;
      // the upper half of a row's chunks lies 128 rows x 128 bytes further on, in the
      // same banks: those lanes take the neighbouring row, whose chunks are permuted
      // to the other banks
      const int r = (tid / CPR) ^ (CPR == 8 ? c >> 2 : 0);
      const uint32_t off0 = (c >> 2) * (BN * 128) + sw128_offset(r, (2 * c) & 7);
      const uint32_t off1 = (c >> 2) * (BN * 128) + sw128_offset(r, (2 * c + 1) & 7);
      const size_t lane_off = static_cast<size_t>(r & 15) * D + c * 16;
      // The codes come one tile ahead, by asynchronous copies into a place of this
      // thread's own, which only it reads back. (Ahead in registers they were no faster
      // than loads waited for at once: 5200 clocks a tile.)
      const uint32_t raw0 = smem_addr(sRaw) + tid * 16;
      auto fetch = [&](int kv, int i, int run) {  // tile i's codes of K or V
        if (i < n) {
          const int key0 = kr.tile(t_beg + i) * BN;
          const bool whole = whole_tile(key0);
          const uint8_t* src = static_cast<const uint8_t*>(kv ? p.pool.v : p.pool.k) + lane_off;
#pragma unroll
          for (int k = 0; k < STEPS; ++k) {
            const int row = r + k * RPS;
            const int at = __shfl_sync(0xffffffffu, run, row >> 4);
            bool valid = at >= 0;
            if (!whole) valid = valid && kr.some_row_sees(key0 + row);
            cp_async16(raw0 + (kv * STEPS + k) * 2048, src + static_cast<size_t>(at < 0 ? 0 : at) * (16 * D), valid);
          }
        }
        cp_async_commit();
      };
      {
        const int run = run_of(0, pg);
        fetch(0, 0, run);
        fetch(1, 0, run);
      }
      for (int i = 0; i < n && ok; ++i) {
        const int pg2 = page_for(i + 2);
        const float ks1 = scale_for(p.pool.k_scale, pg1), vs1 = scale_for(p.pool.v_scale, pg1);
        // V's scale without its exponent, for the 16 keys of lane g
        const float mant = vs * power_of_two(-scale_exponent(vs));
        const bool plain = __all_sync(0xffffffffu, lane >= 8 || mant == 1.f);
        const int run1 = run_of(i + 1, pg1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          cp_async_wait<1>();  // this buffer's copies; the other's may be in flight
          uint4 buf[STEPS];
#pragma unroll
          for (int k = 0; k < STEPS; ++k)
            buf[k] = *reinterpret_cast<const uint4*>(sRaw + (kv * STEPS + k) * 2048 + tid * 16);
          wait_empty(st, round);
          if (!ok) break;
          uint8_t* dst = sKV + st * TILE;
#pragma unroll
          for (int k = 0; k < STEPS; ++k) {
            const uint32_t w[4] = {buf[k].x, buf[k].y, buf[k].z, buf[k].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_f16(w[e], h[2 * e], h[2 * e + 1]);
            if (kv && !plain) {  // a scale that is no power of two
              const __half2 f2 = __float2half2_rn(__shfl_sync(0xffffffffu, mant, (r + k * RPS) >> 4));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h[e]), f2);
                h[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            *reinterpret_cast<uint4*>(dst + off0 + k * (RPS * 128)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + off1 + k * (RPS * 128)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          if (kv == 0) put_meta(i);
          publish(st);
          // the copy into a place that was just read: behind the reads' last use
          fetch(kv, i + 1, run1);
          if (++st == STAGES) st = 0, ++round;
        }
        pg = pg1;
        pg1 = pg2;
        ks = ks1;
        vs = vs1;
      }
      cp_async_wait<0>();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ MMA issuer
    regs_dec<TR::REGS_MMA>();
    if (warp == 4 && n > 0) {
      // The whole warp walks the loop, so that its control flow and the descriptors
      // are uniform, and one elected lane issues. (A loop of one lane's own, under a
      // divergent branch, took 9000 clocks a tile.)
      constexpr uint32_t idS = idesc_dense(BM, BN, TR::FMT, false, false);
      constexpr uint32_t idO = idesc_dense(BM, D, TR::FMT, false, true);
      const uint32_t hi = desc_words(0, 0, 1024, 2).hi;
      const uint32_t q_lo = desc_words(smem_addr(sQ), 16, 1024, 2).lo;
      const uint32_t k_lo = desc_words(smem_addr(sKV), 16, 1024, 2).lo;
      const uint32_t v_lo = desc_words(smem_addr(sKV), BN * 128, 1024, 2).lo;
      const bool leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, s_abort)) != 0;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) mma_commit(bar);
      };
      auto issue_s = [&](int w, int st) {
        const DescWords q{q_lo + w * (TR::QS * TILE >> 4), hi}, kd{k_lo + st * (TILE >> 4), hi};
        const uint32_t d = tbase + TR::S_COL + w * BN;
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * (BM * 128) + (k & 3) * 32;
            mma_bf16_ss(d, desc_at(q, off), desc_at(kd, off), idS, k > 0);
          }
          if constexpr (TR::QS == 2) {  // the second terms of what is rotated
            const DescWords q2{q.lo + (TILE >> 4), hi};
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              if (k * 16 < p.rope.rot) mma_bf16_ss(d, desc_at(q2, k * 32), desc_at(kd, k * 32), idS, true);
          }
          mma_commit(&s_full[w]);
        }
      };
      auto issue_pv = [&](int w, int h, int st, bool first, bool last) {
        const DescWords v{v_lo + st * (TILE >> 4) + h * (TR::HN * 128 >> 4), hi};
        const uint32_t d = tbase + TR::O_COL + w * D, a = tbase + TR::S_COL + w * BN + h * (TR::HN / 2);
        if (leader) {
#pragma unroll
          for (int k = 0; k < TR::HN / 16; ++k)
            mma_bf16_ts(d, a + k * 8, desc_at(v, k * 16 * 128), idO, !first || k > 0);
          if (last) mma_commit(&o_done[w]);
        }
      };
      const int tiles = two ? 2 : 1;
      bool ok = wait(q_full, 0) && wait(&full[0], 0);
      if (ok) {
        tc_fence_after();
        for (int w = 0; w < tiles; ++w) issue_s(w, 0);
        commit(&empty[0]);
      }
      int st = 1, round = 0;  // buffer of V_i and its use
      for (int i = 0; ok && i < n; ++i) {
        const bool more = i + 1 < n;
        if (!(ok = wait(&full[st], round & 1))) break;
        const int v_st = st;
        if (++st == STAGES) st = 0, ++round;
        for (int w = 0; w < tiles; ++w) {
          for (int h = 0; ok && h < 2; ++h) {
            if (!(ok = wait(&p_ready[2 * w + h], i & 1))) break;
            tc_fence_after();
            issue_pv(w, h, v_st, i == 0 && h == 0, !more && h == 1);
          }
          if (!ok) break;
          // V_i's last use: before the next S, whose products would hold its buffer longer
          if (w == tiles - 1) commit(&empty[v_st]);
          if (!more) continue;
          if (w == 0) {
            if (!(ok = wait(&full[st], round & 1))) break;
            tc_fence_after();
          }
          issue_s(w, st);
        }
        if (!ok) break;
        if (more) {
          commit(&empty[st]);
          if (++st == STAGES) st = 0, ++round;
        }
      }
      commit(drain);
      mbar_wait_teardown(drain, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<TR::REGS_SOFTMAX>();
    const int w = (warp - 8) >> 2;
    const int row = (threadIdx.x - 256) & 127;  // TMEM lane
    const int ur = r0 + w * BM + row;           // row of the unit's sequence and head
    const bool live = ur < rows;
    if (w == 0 || two) {
      const int tok = ur / p.group, h = hkv * p.group + ur % p.group;
      const int pos = s.first_pos + tok;
      // ---- this row of Q, rotated, into the operand layout
      float qf = 1.f;
      {
        const __nv_bfloat16* src = p.q + static_cast<long long>(s.q0 + (live ? tok : 0)) * p.q_stride + h * D;
        uint8_t* dst = sQ + w * (TR::QS * TILE);
        uint4 raw[D / 8];  // the whole row in flight at once
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          int lo, hi;
          item_chunks(p.rope, c, lo, hi);
          raw[2 * c] = live ? *reinterpret_cast<const uint4*>(src + lo * 8) : make_uint4(0u, 0u, 0u, 0u);
          raw[2 * c + 1] = live ? *reinterpret_cast<const uint4*>(src + hi * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
        float inv = 1.f;
        if constexpr (E4M3) {  // fp16 under a power of two (see the decode kernel); a rotated element is below 2 amp max
          __nv_bfloat162 a2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) a2 = bf16_amax(raw[c], a2);
          float a = fmaxf(__low2float(a2), __high2float(a2));
          if (p.rope.rot > 0) a *= fmaxf(fabsf(p.rope.amp), 1.f);
          qf = power_below(a);
          inv = 1.f / qf;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          int lo, hi;
          item_chunks(p.rope, c, lo, hi);
          float x[8], y[8];
          unpack8(raw[2 * c], x);
          unpack8(raw[2 * c + 1], y);
          if (c < (p.rope.rot >> 4)) {
            float2 cs[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = turn_fast(p.rope, pos, c * 8 + e);
            rotate_item(p.rope, x, y, cs, 1);
            if constexpr (TR::QS == 2) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = pack_bf16_rest(x[2 * e], x[2 * e + 1]);
                v[4 + e] = pack_bf16_rest(y[2 * e], y[2 * e + 1]);
              }
              *reinterpret_cast<uint4*>(dst + TILE + sw128_offset(row, lo)) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(dst + TILE + sw128_offset(row, hi)) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
          uint32_t u[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u[e] = E4M3 ? pack_f16(x[2 * e] * inv, x[2 * e + 1] * inv) : pack_bf16(x[2 * e], x[2 * e + 1]);
            u[4 + e] = E4M3 ? pack_f16(y[2 * e] * inv, y[2 * e + 1] * inv) : pack_bf16(y[2 * e], y[2 * e + 1]);
          }
          *reinterpret_cast<uint4*>(dst + (lo >> 3) * (BM * 128) + sw128_offset(row, lo & 7)) =
              make_uint4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<uint4*>(dst + (hi >> 3) * (BM * 128) + sw128_offset(row, hi & 7)) =
              make_uint4(u[4], u[5], u[6], u[7]);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      // ---- the keys this row sees: [0, sees_a) and [sees_b, sees_e)
      int sees_a = 0, sees_b = 0, sees_e = 0;
      if (live) {
        sees_e = max(min(pos + 1, s.len), 0);
        sees_b = min(window_begin(p.sc, pos), sees_e);
        const int sink = p.sc.window > 0 ? min(p.sc.n_sink, sees_e) : 0;
        sees_a = max(kr.prefix, sink);
      }
      // positions of this tile's first and last row, for tiles that need no mask
      const int w_lo = s.first_pos + (r0 + w * BM) / p.group;
      const int w_hi = s.first_pos + (min(r0 + w * BM + BM, rows) - 1) / p.group;
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = tbase + lane_off + TR::S_COL + w * BN;
      const uint32_t tO = tbase + lane_off + TR::O_COL + w * D;
      const float fac = qf * p.sc.pre;
      const float slope = MODS & kBiased ? p.sc.slope2[h] : 0.f;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&meta_full[i % TR::META], (i / TR::META) & 1, s_abort));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], i & 1, s_abort));
        if (!ok) break;
        tc_fence_after();
        const KeyGroup* kg = meta + (i % TR::META) * 8;
        const unsigned mapped = static_cast<unsigned>(meta_mapped[i % TR::META]);
        const int key0 = kr.tile(t_beg + i) * BN;
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32(tS + c * 32, sr[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load_wait(sr[c]);
        const bool all_seen = mapped == 255u && (key0 + BN <= kr.prefix ||
                                                 (key0 + BN - 1 <= w_lo && key0 + BN <= s.len &&
                                                  (p.sc.window == 0 || w_hi - key0 < p.sc.window)));
        if constexpr (MODS != 0) {
          const float away = MODS & kBiased ? offset_of(pos, key0) : 0.f;  // of key 0 of the tile
          with_cap<MODS>(p.sc, [&](auto wide) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                sr[c][e] = __float_as_uint(score2<MODS, decltype(wide)::value>(
                    p.sc, __uint_as_float(sr[c][e]), E4M3 ? fac * kg[2 * c + (e >> 4)].ks : fac, slope,
                    away - static_cast<float>(c * 32 + e)));
          });
        }
        if (!all_seen) {
          // 32 keys' visibility as bits, a test and a select per score (with conditions
          // joined by && and || a masked tile took four times an open one)
          auto below = [](int x) { return x <= 0 ? 0u : (x >= 32 ? ~0u : (1u << x) - 1u); };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = key0 + c * 32;
            unsigned seen = below(sees_a - k0) | (below(sees_e - k0) & ~below(sees_b - k0));
            seen &= (mapped >> (2 * c) & 1u ? 0xFFFFu : 0u) | (mapped >> (2 * c + 1) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int e = 0; e < 32; ++e) sr[c][e] = seen & (1u << e) ? sr[c][e] : __float_as_uint(-INFINITY);
          }
        }
        // factors on the scores of the groups (kept off 0, so that masked ones stay -inf)
        // and the exponents of their V scales, read once
        float fg[8], cg[8];
        if constexpr (E4M3)
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float2 u = *reinterpret_cast<const float2*>(kg + g);  // ks, c
            fg[g] = MODS != 0 ? 1.f : fmaxf(fac * u.x, 1e-37f);
            cg[g] = u.y;
          }
        const float f_all = MODS != 0 ? 1.f : fac;  // bf16: one factor
        float mg[8];  // maxima of the groups, chains of their own
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint32_t* v = &sr[g >> 1][(g & 1) * 16];
          float q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            q[e] = fmax3(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                         fmaxf(__uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3])));
          mg[g] = fmaxf(fmax3(q[0], q[1], q[2]), q[3]);
          if constexpr (E4M3) mg[g] = fmaf(mg[g], fg[g], cg[g]);
        }
        float mx = fmaxf(fmax3(fmax3(mg[0], mg[1], mg[2]), mg[3], mg[4]), fmax3(mg[5], mg[6], mg[7]));
        if (!E4M3) mx *= f_all;
        const bool raise = mx > m + (8.f + HEAD);
        const float m_use = raise ? mx - HEAD : m;
        // S_i complete implies that P V i - 1, issued before it, is
        if (__any_sync(0xffffffffu, raise) && i > 0) {
          const float al = raise ? ex2(m - m_use) : 1.f;
          l *= al;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_load32(tO + c * 32, o);
            tmem_load_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
            tmem_store32(tO + c * 32, o);
          }
        }
        m = m_use;
        const float ms = m == -INFINITY ? 0.f : m;
        uint64_t l2 = 0ull;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int g = 2 * c + hf;
            const float f = E4M3 ? fg[g] : f_all, off = E4M3 ? cg[g] - ms : -ms;
            const uint64_t f2 = f2_pack(f, f), off2 = f2_pack(off, off);
            uint64_t part[2] = {0ull, 0ull};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = hf * 16 + 2 * e;
              const uint64_t x2 =
                  f2_fma(f2_pack(__uint_as_float(sr[c][at]), __uint_as_float(sr[c][at + 1])), f2, off2);
              float x0, x1;
              f2_unpack(x2, x0, x1);
              const float e0 = ex2(x0), e1 = ex2(x1);
              part[e & 1] = f2_add(part[e & 1], f2_pack(e0, e1));
              sr[c][hf * 8 + e] = E4M3 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
            }
            const uint64_t sum = f2_add(part[0], part[1]);
            if constexpr (E4M3) l2 = f2_fma(sum, f2_pack(kg[g].share, kg[g].share), l2);
            else l2 = f2_add(l2, sum);
          }
          tmem_store16(tS + c * 16, *reinterpret_cast<uint32_t(*)[16]>(&sr[c][0]));
          if (c & 1) {  // 64 keys of P are on their way
            tmem_store_wait();
            tc_fence_before();
            mbar_arrive(&p_ready[2 * w + (c >> 1)]);
          }
        }
        float u0, u1;
        f2_unpack(l2, u0, u1);
        l += u0 + u1;
      }
      // ---- epilogue
      if (n > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[w], 0, s_abort));
      tc_fence_after();
      m += static_cast<float>(kSumUnit<E4M3>);  // O below: times UNIT
      if (ok) {
        const size_t at = static_cast<size_t>(s.q0 + tok) * p.Hq + h;
        const bool none = m == -INFINITY;
        const float inv = none ? 0.f : 1.f / l;
        if (pieces == 1) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            if (n > 0) {
              tmem_load32(tO + c * 32, o);
              tmem_load_wait(o);
            }
            uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + c * 32);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t u[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = none ? 0u : pack_bf16(__uint_as_float(o[q * 8 + 2 * e]) * UNIT * inv,
                                             __uint_as_float(o[q * 8 + 2 * e + 1]) * UNIT * inv);
              if (live) dst[q] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            __syncwarp();
          }
          if (live && p.lse != nullptr) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_load32(tO + c * 32, o);
            tmem_load_wait(o);
            float4* dst = reinterpret_cast<float4*>(p.part_o + (at * p.nsplit + split) * D + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (live)
                __stcg(dst + q, none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                     : make_float4(__uint_as_float(o[4 * q]) * UNIT, __uint_as_float(o[4 * q + 1]) * UNIT,
                                                   __uint_as_float(o[4 * q + 2]) * UNIT,
                                                   __uint_as_float(o[4 * q + 3]) * UNIT));
            __syncwarp();
          }
          if (live) __stcg(p.part_ml + at * p.nsplit + split, make_float2(m, l));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tbase, TR::TMEM_COLS);
  }
}

}  // namespace ll
