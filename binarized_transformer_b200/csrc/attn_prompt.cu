// attn_prompt.cu -- attention of many new tokens of each sequence over the paged
// key-value cache, on the fifth-generation tensor cores.
//
// S = Q K^T and O = P V with P = 2^(S c - m), c = softmax_scale * log2(e). The rows
// of a tile of 128 are R = 128 / G tokens times the G query heads that share a key
// head, so keys and values are fetched (and E4M3 ones converted) once for all of
// them, and a tile with many shared heads spans few positions: little of it is
// hidden at the diagonal. A block owns two such tiles of one sequence and key head
// and walks their visible key tiles of 128 tokens; the tensor cores work on one
// tile's products while the other tile's softmax runs.
//
// The running reference m of a row starts 7 below its maximum and follows it only when a
// score passes it by more than 15 (ATTN_HEAD, ATTN_SLACK): until then weights up to 2^15 (of
// fp16's 2^16) are kept, and the output in TMEM does not have to be rescaled. Sums and outputs are fp32; P is
// rounded to fp16, its sum is not.
//
// Warps: 0 and 1 issue the MMAs of tile 0 and 1 (the lowest warps of their SM
// sub-partitions, which the others' arithmetic then holds up least), 2 fetches Q (TMA);
// then 4 (E4M3: 8) bring keys and values into shared memory (fp16: asynchronous 16-byte copies; E4M3:
// bulk copies, converted and scaled, exact in fp16); the last 8 are the softmax of tiles
// 0 and 1, a thread a row. A step's keys are taken by halves of 64: the scores of the
// next step's half are computed as soon as this one's weights, which overwrite the
// scores in TMEM (A operand of the second product), have met V. Keys and values lie in
// the same layout (128 rows of 64 values, 128-byte swizzle, one after another for each
// 64 of D): K is read along D, V across it (MN-major).
//
// Few rows (fewer pairs of tiles than half the SMs): clusters of up to 8 blocks share
// the key tiles of a pair; each keeps its unnormalised outputs in shared memory and all
// add them up, some rows each, in the order of the blocks.
//
// Rows of the cache that no row of the block sees are zeros in shared memory (a weight
// of 0 times a NaN would be one). Every wait is bounded; on a
// timeout the block flags it, lets its copies and MMAs finish, frees TMEM and returns.
//
// Measured on a B200, call after call: fp16, 2 x 8192 causal tokens, 32 heads of 128: 1.10
// TFLOP in 1.30 ms, 847 TFLOP/s, 0.52 of cuBLAS's burst rate and 0.62 of its sustained one
// (both under the power limit here, SM clock 1.67 GHz; a cool GPU takes 1.13 ms for one).
// An instruction with N = 64 (the scores of a half) takes as long as one with N = 128, 64
// cycles at best: 48 of them a step and pair, 3070 cycles of about 3700 that it takes. Whole
// 128-key scores (32 instructions a step) leave the tensor cores waiting for the softmax
// and were slower in each form tried (of 1.13 on a cool GPU): 1.47 ms in one place, 1.67
// with the weights beside them, 1.37 with two threads a row and the tiles taking turns.
// E4M3, a chunk of 2700 rows at 64 heads on 8 key heads, window 4096: 363 GFLOP in 489 us,
// 742 TFLOP/s, 0.45 of the burst rate; the conversions add to the issue slots (55% taken).
#include <algorithm>

#include "kv.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace bwta {

constexpr int PR_T = 128;           // rows of a tile, tokens of a key tile
// E4M3 takes twice the warps for the keys and values: they convert them.
template <bool E4M3>
struct PrWarps {
  static constexpr int LOAD = E4M3 ? 8 : 4;
  static constexpr int SOFTMAX0 = 4 + LOAD;  // the first softmax warp
  static constexpr int THREADS = (4 + LOAD + 8) * 32;
  // The issuing warps' loop over halves: with the converting warps beside them the shorter
  // code is faster (windowed chunk 543 -> 515 us), without them the longer (2 x 8192 tokens
  // 1246 -> 1210 us).
  static constexpr int MMA_UNROLL = E4M3 ? 1 : 2;
  // Registers by role; launched with 128 (96) a thread, so 4 x 128 (5 x 96) in all.
  static constexpr int REG_MMA = E4M3 ? 56 : 104, REG_LOAD = E4M3 ? 72 : 104;
  static constexpr int REG_SOFTMAX = E4M3 ? 136 : 152;
  static_assert(REG_MMA + LOAD / 4 * REG_LOAD + 2 * REG_SOFTMAX <= (E4M3 ? 5 * 96 : 4 * 128), "registers");
};
// Key or value tiles whose copies a loading warp leaves in flight before it hands one over
// (2 x 8192 tokens: none 1219 us, one 1140, two 1176).
constexpr int PR_LAG = 1;
constexpr int PR_HALF = 64;         // keys of one product (scores and weights)
constexpr int PR_MIN_STEPS = 2;     // key tiles that are worth a block of their own
template <int DP, bool E4M3>
struct PrShape {
  static constexpr int NH = DP / 64;                  // halves of 64 columns
  static constexpr int TILE = NH * PR_T * 128;        // bytes of 128 rows
  static constexpr int SLOTS = DP == 128 ? (E4M3 ? 4 : 5) : 8;  // key and value tiles in the ring
  static constexpr int RAW = E4M3 ? 16 * DP : 0;  // 16 rows as they lie in the cache
  static constexpr int BARS = 1024;
  static constexpr int SMEM = 1024 + (2 + SLOTS) * TILE + 16 * RAW + BARS;
  static_assert(SMEM <= 232448, "shared memory of a block");
};

struct PrArgs {
  AttnArgs a;
  int group, R;      // query heads of a key head, tokens of a tile
  int split;         // blocks (a cluster) that share the key tiles of a pair
};

struct PrItem {
  int64_t row0;        // of the pair's first token
  int32_t slot, head;  // key head
  int32_t cnt[2];      // tokens of each tile
  int32_t pmin[2];     // position of a tile's first token (may be negative)
  int32_t last[2], first[2], sink[2];  // its visible key tiles: [0, sink) and [first, last]; last < 0: none
  // this block's share of the walk over all of them: step j is tile j + j0 below u_sink
  // (tiles among the sinks), j + u_first from there on
  int32_t u_sink, u_first, j0, steps;
  int32_t parts;       // blocks that have one
  int32_t lo, hi;      // tokens that some row sees: [lo, hi] and those below the sinks
  bool live;
};

struct PrBars {
  uint64_t full[8], empty[8], raw[8][2];
  uint64_t q_ready;
  uint64_t s_ready[2][2], p_ready[2][2], pv_done[2], o_done[2], drain[2];
  uint32_t tmem_base;
  int32_t timeout, undrained;
  PrItem item;
};

__device__ __forceinline__ bool pr_wait(PrBars *b, uint64_t *bar, uint32_t parity) {
  // no suspend-time hint: these waits are short and follow one another in a chain
  const uint32_t at = smem_addr(bar);
  uint64_t t0 = 0;
  for (int i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (done) return true;
    if (i % 64 == 63) {
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > 2000000000ull || *(volatile int32_t *)&b->timeout) break;
    }
  }
  b->timeout = 1;
  return false;
}


template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Block -> sequence, key head and pair of tiles. The pairs of a (sequence, head)
// follow one another, the last (longest) first: their blocks run side by side
// and share the keys in L2. Called by one warp.
__device__ __forceinline__ void pr_find(const PrArgs &A, PrItem &it) {
  const AttnArgs &a = A.a;
  const int lane = threadIdx.x % 32;
  const int64_t at = blockIdx.x / A.split, H = a.c.H, two = 2 * A.R;
  int64_t before = 0;
  it.live = false;
  for (int64_t s0 = 0; s0 < a.n_seq; s0 += 32) {
    const int64_t s = s0 + lane;
    int64_t c0 = 0, c1 = 0, len = 0;
    int32_t slot = -1;
    bool bad = false;
    if (s < a.n_seq) {  // all that may be needed of a sequence at once: one latency after another counts
      slot = kv_slot(a.r, s);
      len = kv_length(a.r, slot, a.c.ps, bad);
      c0 = min(max((int64_t)a.cu_q[s], (int64_t)0), a.total_q);
      c1 = min(max((int64_t)a.cu_q[s + 1], c0), a.total_q);
    }
    const int64_t pairs = div_pos(c1 - c0 + two - 1, two);
    int64_t x = pairs * H;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t y = __shfl_up_sync(FULL, x, d);
      if (lane >= d) x += y;
    }
    const unsigned hit = __ballot_sync(FULL, before + x > at);
    if (!hit) {
      before += __shfl_sync(FULL, x, 31);
      continue;
    }
    if (lane == __ffs(hit) - 1) {
      const int64_t local = at - (before + x - pairs * H);
      const int64_t head = div_pos(local, pairs), pair = pairs - 1 - (local - head * pairs);
      const int64_t n = c1 - c0;
      it.slot = slot;
      if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
      it.head = (int32_t)head;
      it.row0 = c0 + pair * two;
      it.j0 = it.steps = 0;
      it.parts = 1;
      int64_t pmax_all = -1, pmin_all = 0;
      int32_t u_last = -1, u_first = 0x7fffffff, u_sink = 0;
      for (int i = 0; i < 2; ++i) {
        const int64_t tok = pair * two + i * A.R;
        const int64_t cnt = min(max(n - tok, (int64_t)0), (int64_t)A.R);
        const int64_t pmin = len - n + tok, pmax = pmin + cnt - 1;
        it.cnt[i] = (int32_t)cnt;
        it.pmin[i] = (int32_t)max(pmin, (int64_t)-256);  // 256 rows at most follow: all of them negative
        it.last[i] = -1;
        it.first[i] = it.sink[i] = 0;
        if (cnt == 0 || pmax < 0) continue;
        const int64_t lo = a.window ? max((int64_t)0, pmin - a.window + 1) : 0;
        it.last[i] = (int32_t)(pmax / PR_T);
        it.first[i] = (int32_t)(lo / PR_T);
        it.sink[i] = (int32_t)min((a.sinks + PR_T - 1) / PR_T, lo / PR_T);
        if (u_last < 0) pmin_all = pmin;
        pmax_all = pmax;
        u_last = max(u_last, it.last[i]);
        u_first = min(u_first, it.first[i]);
        u_sink = max(u_sink, it.sink[i]);
      }
      if (u_last >= 0) {
        u_sink = min(u_sink, u_first);
        const int all = u_sink + u_last - u_first + 1, rank = blockIdx.x % A.split;
        it.parts = max(1, min(A.split, all / PR_MIN_STEPS));
        it.j0 = rank < it.parts ? (int)((int64_t)all * rank / it.parts) : 0;
        it.steps = rank < it.parts ? (int)((int64_t)all * (rank + 1) / it.parts) - it.j0 : 0;
        it.u_sink = u_sink - it.j0;
        it.u_first = u_first - it.u_sink;
        it.lo = (int32_t)(a.window ? max((int64_t)0, pmin_all - a.window + 1) : 0);
        it.hi = (int32_t)pmax_all;
      }
      it.live = true;
    }
    return;
  }
}

// Eight E4M3 bytes as halves times their row's scale (both exact in fp16).
__device__ __forceinline__ uint4 pr_convert(uint2 b, uint32_t scale2) {
  auto four = [&](uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 a, b;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 a, l;\n\tcvt.rn.f16x2.e4m3x2 b, h;\n\t"
        "mul.rn.f16x2 %0, a, %3;\n\tmul.rn.f16x2 %1, b, %3;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x), "r"(scale2));
  };
  uint4 v;
  four(b.x, v.x, v.y);
  four(b.y, v.z, v.w);
  return v;
}

// The lowest n bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

__device__ __forceinline__ float pr_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two numbers as halves, those past fp16's range as +-65504 (NaN stays). Rounded weights
// over the sum of unrounded ones make means up to 2^-11 larger than the largest value.
__device__ __forceinline__ uint32_t pr_half2_limited(float x, float y) {
  uint32_t h;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  return h;
}

// Two fp32 numbers in a register pair: one instruction for both.
__device__ __forceinline__ uint64_t pk2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 up2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int DP, bool E4M3>
__global__ void __launch_bounds__(PrWarps<E4M3>::THREADS, 1) k_attn_prompt(const __grid_constant__ CUtensorMap map_q, const PrArgs A) {
  using S = PrShape<DP, E4M3>;
  using W = PrWarps<E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  PrBars *bars = reinterpret_cast<PrBars *>(base + (2 + S::SLOTS) * S::TILE + 16 * S::RAW);
  static_assert(sizeof(PrBars) <= S::BARS, "barriers");
  const AttnArgs &a = A.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, D = a.c.D;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&bars->full[i], W::LOAD);
      mbar_init(&bars->empty[i], 2);
    }
    mbar_init(&bars->q_ready, 1);
    prefetch_tensormap(&map_q);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_ready[i][0], 1);
      mbar_init(&bars->s_ready[i][1], 1);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->p_ready[i][0], 4);
      mbar_init(&bars->p_ready[i][1], 4);
      mbar_init(&bars->o_done[i], 1);
      mbar_init(&bars->drain[i], 1);
    }
    for (int i = 0; i < 16; ++i) mbar_init(&bars->raw[i / 2][i % 2], 1);
    bars->timeout = bars->undrained = 0;
    mbar_fence_init();
  }
  if (D % 16 != 0) {  // the products read 8 columns past D, which are never written: zero once
    for (int i = threadIdx.x * 16; i < (2 + S::SLOTS) * S::TILE; i += W::THREADS * 16)
      *reinterpret_cast<uint4 *>(base + i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (A.R * A.group < PR_T) {  // rows that the copies of Q leave out
    for (int i = threadIdx.x * 16; i < 2 * S::TILE; i += W::THREADS * 16)
      *reinterpret_cast<uint4 *>(base + i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 4) pr_find(A, bars->item);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const PrItem &it = bars->item;
  // TMEM columns: S0 0, S1 128, O0 256, O1 384 (P of a tile: the first 64 of its S)
  const int steps = it.live ? it.steps : 0;

  if (warp >= W::SOFTMAX0) {
    // ------------------------------------------------ softmax and output
    regs_inc<W::REG_SOFTMAX>();
    const int w = (warp - W::SOFTMAX0) / 4, q = warp % 4, r = q * 32 + lane;
    if (it.live) {
      const int chunks = D / 8;
      uint8_t *qs = base + w * S::TILE;
      const int used = it.cnt[w] * A.group;
      const uint32_t by_chunks = 65536u / chunks + 1, by_group = 65536u / A.group + 1;  // exact below 2048
      const int tok = r / A.group;
      const int p = it.pmin[w] + tok;
      const bool valid = r < used;
      const int64_t lo64 = a.window ? (int64_t)p - a.window + 1 : 0;
      const int p_min = it.pmin[w], p_max = it.pmin[w] + it.cnt[w] - 1;
      const float c2 = a.scale * 1.44269504088896340736f;
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      uint32_t halves = 0;  // of key tiles, so far
      const uint32_t ts = tmem_addr(tmem, q * 32, w * 128), to = tmem_addr(tmem, q * 32, 256 + w * 128);
      const uint64_t cc = pk2(c2, c2);
      // in registers: every barrier would have them read again
      const int n = steps, j0 = it.j0, u_sink = it.u_sink, u_first = it.u_first;
      const int last = it.last[w], first = it.first[w], sink = it.sink[w];
      for (int j = 0; j < n && ok; ++j) {
        const int t = j + (j < u_sink ? j0 : u_first);  // the key tile
        if (t > last || (t < first && t >= sink)) continue;
        for (int h = 0; h < 2; ++h, ++halves) {
          const int k0 = t * PR_T + h * PR_HALF;
          const bool all = k0 + PR_HALF - 1 <= p_min &&
                           (!a.window || k0 > p_max - a.window || k0 + PR_HALF <= a.sinks);
          ok = __all_sync(FULL, pr_wait(bars, &bars->s_ready[w][h], (halves >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          uint32_t v[2][32];
          tmem_ld32(ts + h * PR_HALF, v[0]);
          tmem_ld32(ts + h * PR_HALF + 32, v[1]);
          tmem_wait_ld();
          if (!all) {
            const int hi = valid ? p - k0 : -1;
            const int lo = (int)min(max(lo64 - k0, (int64_t)0), (int64_t)PR_HALF);
            const int sk = (int)min(max(a.sinks - k0, (int64_t)0), (int64_t)PR_HALF);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t see = below(hi + 1 - c * 32) & (~below(lo - c * 32) | below(sk - c * 32));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1)) v[c][i] = 0xff800000u;
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 4)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              top[c] = fmaxf(fmaxf(top[c], __uint_as_float(v[c / 2][i + (c % 2) * 2])),
                             __uint_as_float(v[c / 2][i + (c % 2) * 2 + 1]));
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          // in one rounding, as the weights below take it; also from -infinity
          const bool up = fmaf(mx, c2, -m) > ATTN_SLACK;
          if (__any_sync(FULL, up)) {
            // From 2^28 on fp32 has steps of 32: no m can then be trusted to leave the largest weight
            // in fp16's range, and the row becomes NaN. (A second rounding step in the loop below
            // would serve such scores; 2 x 8192 tokens 1306 -> 1330 us.)
            float mn = up ? fmaf(mx, c2, -ATTN_HEAD) : m;
            if (fabsf(mn) >= 268435456.0f && up) mn = __int_as_float(0x7fffffff);
            // nothing seen so far: the sums are zero and the factor does not matter
            const float f = m == -INFINITY ? 0.0f : pr_exp2(m - mn);
            m = mn;
            l *= f;
            if (halves > 0) {  // the product before this one is complete: O holds still
              ok = __all_sync(FULL, pr_wait(bars, &bars->pv_done[w], (halves - 1) & 1));
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < DP / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(to + c * 16, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(to + c * 16, o);
              }
            }
          }
          const float z = m == -INFINITY ? 0.0f : m;
          const uint64_t zz = pk2(-z, -z);
          uint64_t sum[2] = {0, 0};
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = i / 16, e = (i % 16) * 2;
            float2 y = up2(fma2(pk2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), cc, zz));
            y.x = pr_exp2(y.x);
            y.y = pr_exp2(y.y);
            sum[i % 2] = add2(sum[i % 2], pk2(y.x, y.y));
            const __half2 two = __floats2half2_rn(y.x, y.y);
            pk[i] = *reinterpret_cast<const uint32_t *>(&two);
          }
          tmem_st32(ts + h * PR_HALF, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_ready[w][h]);
          const float2 sa = up2(add2(sum[0], sum[1]));
          l += sa.x + sa.y;
        }
      }
      // output
      bool finite = true;
      // (for a share, which goes where the keys and values are, both tiles' products)
      if (steps > 0 && ok)
        ok = __all_sync(FULL, pr_wait(bars, &bars->o_done[w], 0) &&
                                  (it.parts == 1 || pr_wait(bars, &bars->o_done[1 - w], 0)));
      if (ok && it.parts > 1 && steps > 0) {
        // a share: for the cluster to add up
        tc_fence_after();
        float *part = reinterpret_cast<float *>(base + 2 * S::TILE) + (w * PR_T + r) * DP;
#pragma unroll 1
        for (int c = 0; c * 32 < D; ++c) {
          uint32_t o[32];
          if (halves > 0) {
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(part + (((c * 8 + i) ^ r) % (DP / 4)) * 4) =
                halves > 0 ? make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]) : make_uint4(0, 0, 0, 0);
        }
        *reinterpret_cast<float2 *>(base + (w * PR_T + r) * 8) = make_float2(m, l);
      } else if (ok && blockIdx.x % A.split == 0) {
        tc_fence_after();
        const bool none = p < 0;  // sees nothing: zeros (from p = 0 on a row sees a key)
        const float inv = 1.0f / l;
        float zero = 0.0f;  // stays 0 unless an output is not finite
        // through shared memory (Q has been read), so that rows are written whole
#pragma unroll 1
        for (int c = 0; c * 32 < D; ++c) {
          uint32_t o[32];
          if (halves > 0) {
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = none ? 0.0f : __uint_as_float(o[i * 8 + 2 * e]) * inv;
              const float y = none ? 0.0f : __uint_as_float(o[i * 8 + 2 * e + 1]) * inv;
              if (c * 32 + i * 8 < D) zero = fmaf(x, 0.0f, fmaf(y, 0.0f, zero));
              h[e] = pr_half2_limited(x, y);
            }
            const int cc = c * 4 + i;
            *reinterpret_cast<uint4 *>(qs + (cc / 8) * (PR_T * 128) + swz128(r, cc % 8)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        finite = !valid || zero == 0.0f;
        if (!finite) {  // the limit has taken Inf too: +-65504 in this row is Inf again
#pragma unroll 1
          for (int i = 0; i < chunks * 4; ++i) {
            uint32_t *h = reinterpret_cast<uint32_t *>(qs + (i / 32) * (PR_T * 128) + swz128(r, i / 4 % 8)) + i % 4;
            *h += (*h & 0x7fffu) == 0x7bffu;
            *h += (*h & 0x7fff0000u) == 0x7bff0000u ? 0x10000u : 0u;
          }
        }
        __syncwarp();
        uint16_t *out = a.out + (it.row0 + (int64_t)w * A.R) * a.ldo + (int64_t)it.head * A.group * D;
#pragma unroll 4
        for (int p = lane; p < 32 * chunks; p += 32) {
          const int r0 = (int)((p * by_chunks) >> 16), c = p - r0 * chunks, rr = q * 32 + r0;
          const int i = (int)((rr * by_group) >> 16);
          const uint4 y = *reinterpret_cast<const uint4 *>(qs + (c / 8) * (PR_T * 128) + swz128(rr, c % 8));
          if (rr < used)
            *reinterpret_cast<uint4 *>(out + (int64_t)i * a.ldo + (int64_t)(rr - i * A.group) * D + c * 8) = y;
        }
      }
      if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ keys and values
    regs_dec<W::REG_LOAD>();
    constexpr int GROUPS = 8 / W::LOAD;  // 16 tokens each, of a tile's 8
    constexpr int ITER = DP / 16;  // 16-byte chunks of fp16 a lane holds of 16 rows
    const int chunks = D / 8, n = 2 * steps;
    const uint32_t recip = 65536u / chunks + 1;  // p / chunks = (p * recip) >> 16 for p < 256
    bool bad = false;
    const uint32_t w2 = warp - 4;
    // in registers: every barrier would have them read again
    const int lo = it.lo, hi = it.hi, j0 = it.j0, u_sink = it.u_sink, u_first = it.u_first;
    const int64_t head_row = (int64_t)it.head * a.c.ps;
    // 16 tokens of key tile j (and their values): the offset of the first (in
    // elements; scales: in floats), which of the 16 rows to read
    struct Place {
      int64_t at, sat;
      uint32_t rows;
    };
    auto token = [&](int j, int gi) {
      return (j + (j < u_sink ? j0 : u_first)) * PR_T + (int)(w2 * GROUPS + gi) * 16;
    };
    // tok / ps, both multiples of 16: the quotient of a multiplication is right or 1 short
    const uint32_t ps16 = a.c.ps / 16, by_ps = 0xffffffffu / ps16;
    const int32_t *row_of_pages = a.r.pages + (int64_t)it.slot * a.r.ld;
    auto split = [&](int tok, int &in) -> int {
      uint32_t n = __umulhi((uint32_t)tok / 16, by_ps), r = (uint32_t)tok / 16 - n * ps16;
      if (r >= ps16) {
        ++n;
        r -= ps16;
      }
      in = (int)r * 16;
      return (int)n;
    };
    // the page's number is fetched a tile ahead
    auto page_of = [&](int j, int gi) -> int32_t {
      const int tok = token(j, gi);
      int in;
      return j < steps && tok <= hi ? row_of_pages[split(tok, in)] : -1;
    };
    auto place = [&](int j, int gi, int32_t page) -> Place {
      const int tok = token(j, gi);
      Place p{0, 0, 0};
      // bit r: token tok + r is seen by some row
      const int top = min(hi - tok + 1, 16);
      if (top <= 0) return p;
      p.rows = (1u << top) - 1;
      if (a.window && tok < lo) {
        const uint32_t win = lo - tok >= 16 ? 0u : 0xffffu << (lo - tok);
        const int64_t sk = a.sinks - tok;
        p.rows &= win | (sk >= 16 ? 0xffffu : sk <= 0 ? 0u : (1u << sk) - 1);
        if (!p.rows) return p;
      }
      if ((uint32_t)page >= (uint32_t)a.c.num_pages) {
        bad = true;
        p.rows = 0;
        return p;
      }
      int in;
      split(tok, in);
      const int64_t row = head_row + in;
      p.at = (int64_t)page * a.c.page_stride + row * D;
      p.sat = (int64_t)page * a.c.scale_stride + row;
      return p;
    };
    auto slot_of = [&](int u) { return base + (2 + u % S::SLOTS) * S::TILE; };
    auto arrive = [&](int u) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->full[u % S::SLOTS]);
    };
    auto dst_of = [&](int gi, int p) -> uint32_t {
      const int r = (int)((p * recip) >> 16), c = p - r * chunks;
      return (uint32_t)((c / 8) * (PR_T * 128)) + swz128((w2 * GROUPS + gi) * 16 + r, c % 8);
    };
    bool ok = true;
    if (!E4M3) {
      Place pl[GROUPS];
      int32_t page[GROUPS];
#pragma unroll
      for (int gi = 0; gi < GROUPS; ++gi) page[gi] = page_of(0, gi);
      for (int u = 0; u < n && ok; ++u) {  // keys and values of a tile in turn
        if (!(u & 1)) {
#pragma unroll
          for (int gi = 0; gi < GROUPS; ++gi) {
            pl[gi] = place(u / 2, gi, page[gi]);
            page[gi] = page_of(u / 2 + 1, gi);
          }
        }
        if (u >= S::SLOTS) ok = pr_wait(bars, &bars->empty[u % S::SLOTS], (u / S::SLOTS - 1) & 1);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        const uint32_t st = smem_addr(slot_of(u));
        const uint16_t *kv = reinterpret_cast<const uint16_t *>(u & 1 ? a.c.v : a.c.k);
#pragma unroll
        for (int gi = 0; gi < GROUPS; ++gi)
#pragma unroll
          for (int i = 0; i < ITER; ++i) {
            const int p = i * 32 + lane;
            if (p < 16 * chunks) {
              const int r = (int)((p * recip) >> 16);
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(st + dst_of(gi, p)),
                           "l"(kv + pl[gi].at + p * 8), "r"((pl[gi].rows >> r) & 1 ? 16 : 0)
                           : "memory");
            }
          }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (u >= PR_LAG) {
          asm volatile("cp.async.wait_group %0;" ::"n"(PR_LAG) : "memory");
          arrive(u - PR_LAG);
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (ok)
        for (int v = max(0, n - PR_LAG); v < n; ++v) arrive(v);
    } else {
      // a ring of this warp's own: 16 rows of keys and 16 of values, each
      // refilled for the next tile as soon as it has been converted
      uint8_t *raw = base + (2 + S::SLOTS) * S::TILE + w2 * 2 * S::RAW;
      int32_t page = page_of(0, 0);
      Place pl;          // of the tile whose copies are under way
      uint32_t rows[2];  // visible ones of the pieces in the ring
      float sc[2] = {0, 0};  // and the scales of their rows (lanes 16 .. 31: again)
      uint32_t fetched[2] = {0, 0};
      auto fetch = [&](int q) {  // piece q: keys (0) or values (1)
        const Place &p = pl;
        rows[q] = p.rows;
        ++fetched[q];
        uint64_t *bar = &bars->raw[w2][q];
        if (p.rows) {
          const uint32_t on = lane == 0;
          mbar_arrive_expect_tx_if(on, bar, 16 * D);
          bulk_load_if(on, raw + q * S::RAW, (q == 0 ? a.c.k : a.c.v) + p.at, 16 * D, bar);
          sc[q] = (q == 0 ? a.c.ks : a.c.vs)[p.sat + (lane & 15)];
        } else if (lane == 0) {
          mbar_arrive(bar);
        }
      };
      auto places = [&](int j) {
        pl = place(j, 0, page);
        page = page_of(j + 1, 0);
      };
      if (steps > 0) {
        places(0);
#pragma unroll
        for (int q = 0; q < 2; ++q) fetch(q);
      }
      int j = 0;
      for (; j < steps && ok; ++j) {
        if (j + 1 < steps) places(j + 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = 2 * j + q;
          bool fine = true;
          if (u >= S::SLOTS) fine = pr_wait(bars, &bars->empty[u % S::SLOTS], (u / S::SLOTS - 1) & 1);
          fine = fine && pr_wait(bars, &bars->raw[w2][q], j & 1);
          ok = __all_sync(FULL, fine);
          if (!ok) break;
          uint8_t *st = slot_of(u);
          const uint8_t *from = raw + q * S::RAW;
          uint32_t one = (uint32_t)__half_as_ushort(__float2half_rn(sc[q]));
          one |= one << 16;
          if (D == DP && rows[q] == 0xffffu) {
            // all loads, then all stores: nothing waits for a piece by itself
            constexpr int C = DP / 8;  // chunks of a row
            uint2 x[ITER];
#pragma unroll
            for (int i = 0; i < ITER; ++i) x[i] = *reinterpret_cast<const uint2 *>(from + (i * 32 + lane) * 8);
            uint8_t *to = st + ((lane % C) / 8) * (PR_T * 128);
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
              const int r = i * (32 / C) + lane / C;
              *reinterpret_cast<uint4 *>(to + (w2 * 16 * 128) + swz128(r, lane % 8)) =
                  pr_convert(x[i], __shfl_sync(FULL, one, r));
            }
          } else {
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
              const int p = i * 32 + lane, r = (int)((p * recip) >> 16) & 15;
              const uint32_t s2 = __shfl_sync(FULL, one, r);
              if (p < 16 * chunks) {
                uint4 x = pr_convert(*reinterpret_cast<const uint2 *>(from + p * 8), s2);
                if (!((rows[q] >> r) & 1)) x = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(st + dst_of(0, p)) = x;
              }
            }
          }
          __syncwarp();  // the piece has been read
          if (j + 1 < steps) fetch(q);
          arrive(u);
        }
      }
      if (!ok && lane == 0)  // copies under way land before the block ends
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (!mbar_wait(&bars->raw[w2][q], (fetched[q] - 1) & 1, DRAIN_NS)) bars->undrained = 1;
    }
    if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
  } else {
    // ------------------------------------------------ MMA issue
    regs_dec<W::REG_MMA>();
    // warp 2: the rows of Q, R tokens of G heads, into the layout of the keys (rows past the
    // tile's are other tokens' and do not count)
    if (warp == 2 && lane == 0 && steps > 0) {
      const uint32_t bytes = 128 * A.R * A.group;
      const int tiles = it.cnt[1] > 0 ? 2 : 1;
      mbar_arrive_expect_tx(&bars->q_ready, tiles * S::NH * bytes);
      for (int i = 0; i < tiles * S::NH; ++i)
        tma_load_3d(base + i / S::NH * S::TILE + i % S::NH * (PR_T * 128), &map_q, i % S::NH * 64,
                    it.head * A.group, (int32_t)it.row0 + i / S::NH * A.R, &bars->q_ready);
      if (!mbar_wait(&bars->q_ready, 0)) bars->timeout = bars->undrained = 1;
    }
    // warp w issues the products of tile w, all lanes in step
    if (warp < 2 && steps > 0) {
      const int w = warp, n = __shfl_sync(FULL, steps, 0);
      const uint32_t on = lane == 0;
      const uint32_t id_qk = idesc_f16_f32(PR_T, PR_HALF);
      const uint32_t id_pv = idesc_f16_f32(PR_T, (D + 15) / 16 * 16) | IDESC_B_MN;
      const int ks = (D + 15) / 16;
      const uint32_t s0 = __shfl_sync(FULL, smem_addr(base), 0);
      const uint32_t ts = __shfl_sync(FULL, tmem, 0) + w * 128, to = ts + 256;
      const uint64_t qa = smem_desc_k_sw128(s0 + w * S::TILE);
      const uint64_t ring_k = smem_desc_k_sw128(s0 + 2 * S::TILE);
      const uint64_t ring_mn = smem_desc_mn_sw128(s0 + 2 * S::TILE, PR_T * 128);
      const int last = __shfl_sync(FULL, it.last[w], 0), first = __shfl_sync(FULL, it.first[w], 0);
      const int sink = __shfl_sync(FULL, it.sink[w], 0);
      const int u_sink = __shfl_sync(FULL, it.u_sink, 0), u_first = __shfl_sync(FULL, it.u_first, 0);
      const int j0 = __shfl_sync(FULL, it.j0, 0);
      auto active = [&](int j) {
        const int t = j + (j < u_sink ? j0 : u_first);
        return t <= last && (t >= first || t < sink);
      };
      auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, pr_wait(bars, bar, parity)); };
      struct Ring {
        int slot;
        uint32_t phase;
        __device__ void next() {
          if (++slot == S::SLOTS) {
            slot = 0;
            phase ^= 1;
          }
        }
      };
      Ring ring = {0, 0};
      uint32_t p_phase = 0, more = 0;
      auto qk = [&](int slot, int h) {
        const uint64_t kb = ring_k + (uint64_t)((slot * S::TILE + h * PR_HALF * 128) >> 4);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          if (k >= ks) break;
          const uint32_t off = ((k / 4) * (PR_T * 128) + (k % 4) * 32) >> 4;
          mma_f16_ss_if(on, ts + h * PR_HALF, qa + off, kb + off, id_qk, k > 0);
        }
        tc_commit_if(on, &bars->s_ready[w][h]);
      };
      bool ok = ready(&bars->q_ready, 0) && ready(&bars->full[0], 0);
      if (ok) {
        tc_fence_after();
        if (active(0)) {
          qk(0, 0);
          qk(0, 1);
        }
        tc_commit_if(on, &bars->empty[0]);
        ring.next();
      }
      // Both tiles of keys and values that a step needs are waited for ahead of the
      // weights, and nothing stands between the weights of a half and the next scores
      // in its place.
      for (int j = 0; j < n && ok; ++j) {
        const int sv = ring.slot;  // the values of step j, then the keys of step j + 1
        ok = ready(&bars->full[sv], ring.phase);
        ring.next();
        const int sk = ring.slot;
        const bool go = active(j), go_on = j + 1 < n && active(j + 1);
        if (j + 1 < n) ok = ok && ready(&bars->full[sk], ring.phase);
        const uint64_t vb = ring_mn + (uint64_t)(sv * (S::TILE >> 4));
        if (!ok) break;
        tc_fence_after();
#pragma unroll W::MMA_UNROLL
        for (int h = 0; h < 2; ++h) {
          if (go) {
            ok = ok && ready(&bars->p_ready[w][h], p_phase);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mma_f16_ts_if(on, to, ts + h * PR_HALF + k * 8, vb + (uint64_t)((h * 4 + k) * (2048 >> 4)), id_pv, more);
              more = 1;
            }
            tc_commit_if(on, &bars->pv_done[w]);
          }
          if (go_on) qk(sk, h);
        }
        if (!ok) break;
        if (go) p_phase ^= 1;
        tc_commit_if(on, j + 1 == n ? &bars->o_done[w] : &bars->empty[sv]);
        if (j + 1 < n) tc_commit_if(on, &bars->empty[sk]);
        ring.next();
      }
      // every MMA has completed before TMEM is released
      tc_commit_if(on, &bars->drain[w]);
      if (!mbar_wait(&bars->drain[w], 0, DRAIN_NS)) bars->undrained = 1;
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (A.split > 1) {
    // Shares of one pair: every block adds up some of its rows, o = sum_k o_k f_k / sum_k l_k f_k
    // with f_k = 2^(m_k - max m), reading the others' shared memory.
    cluster_sync();
    const int parts = it.parts, rank = blockIdx.x % A.split;
    if (it.live && parts > 1 && rank < parts && warp >= W::SOFTMAX0) {
      bool finite = true;
      const uint32_t ml0 = smem_addr(base), o0 = smem_addr(base + 2 * S::TILE);
      for (int i = (warp - W::SOFTMAX0) * parts + rank; i < 2 * PR_T; i += 8 * parts) {
        const int w = i / PR_T, r = i % PR_T;
        if (r >= it.cnt[w] * A.group) continue;
        float M = -INFINITY, L = 0.0f;
        float4 y = make_float4(0, 0, 0, 0);
        for (int k = 0; k < parts; ++k) M = fmaxf(M, cluster_ld2(ml0 + i * 8, k).x);
        for (int k = 0; k < parts; ++k) {
          const float2 ml = cluster_ld2(ml0 + i * 8, k);
          const float f = ml.x == -INFINITY ? 0.0f : pr_exp2(ml.x - M);
          L += ml.y * f;
          const float4 x = cluster_ld4(o0 + (i * DP + ((lane ^ r) % (DP / 4)) * 4) * 4, k);
          y.x += x.x * f;
          y.y += x.y * f;
          y.z += x.z * f;
          y.w += x.w * f;
        }
        if (lane * 4 < D) {
          const int tok = r / A.group;
          const bool none = it.pmin[w] + tok < 0;  // sees nothing: zeros
          const float inv = 1.0f / L;
          float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[e] = none ? 0.0f : mean_to_f16_range(z[e] * inv);
            finite &= z[e] - z[e] == 0.0f;
          }
          const __half2 a2 = __floats2half2_rn(z[0], z[1]), b2 = __floats2half2_rn(z[2], z[3]);
          uint16_t *out = a.out + (it.row0 + (int64_t)w * A.R + tok) * a.ldo +
                          ((int64_t)it.head * A.group + (r - tok * A.group)) * D;
          *reinterpret_cast<uint2 *>(out + lane * 4) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&a2), *reinterpret_cast<const uint32_t *>(&b2));
        }
      }
      if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its shares are read
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && bars->timeout)
    flag_status(a.d_status, BWTA_STATUS_TIMEOUT | (bars->undrained ? BWTA_STATUS_DRAIN : 0));
}

int64_t attn_prompt_blocks(int64_t n_seq, int64_t total_q, int64_t n_heads, int64_t n_kv_heads) {
  const int64_t two = 2 * (PR_T / (n_heads / n_kv_heads));
  return n_kv_heads * (total_q / two + std::min(n_seq, total_q));  // a sum of rounded-up quotients at most
}

// Q as [total_q][n_heads][D]; a box is 64 columns of a tile's tokens and heads.
static bool make_q_map(CUtensorMap *map, const PrArgs &A) {
  PFN_encodeTiled enc = get_encode_tiled();
  if (!enc) return false;
  const AttnArgs &a = A.a;
  cuuint64_t dims[3] = {(cuuint64_t)a.c.D, (cuuint64_t)a.n_heads, (cuuint64_t)a.total_q};
  cuuint64_t strides[2] = {(cuuint64_t)a.c.D * 2, (cuuint64_t)a.ldq * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)A.group, (cuuint32_t)A.R};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool E4M3>
static cudaError_t launch_prompt_t(const PrArgs &A, int64_t blocks, cudaStream_t s) {
  static SmemOptIn opt_in;
  auto kern = k_attn_prompt<DP, E4M3>;
  if (cudaError_t e = opt_in(kern, PrShape<DP, E4M3>::SMEM)) return e;
  CUtensorMap map;
  if (!make_q_map(&map, A)) return cudaErrorInvalidValue;
  return launch_pdl_cluster(kern, dim3((unsigned)(blocks * A.split)), (unsigned)A.split, dim3(PrWarps<E4M3>::THREADS),
                            PrShape<DP, E4M3>::SMEM, s, map, A);
}

cudaError_t launch_attn_prompt(const AttnArgs &a, bool e4m3, cudaStream_t s) {
  PrArgs A = {};
  A.a = a;
  A.group = a.n_heads / a.c.H;
  A.R = PR_T / A.group;
  const int64_t blocks = attn_prompt_blocks(a.n_seq, a.total_q, a.n_heads, a.c.H);
  // Few pairs leave SMs idle: up to 8 blocks then share the keys of each.
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // (As many as the longest walk that the table allows has shares for; measured: 3 rows
  // over 8000 tokens 129 -> 23 us, while shares of nothing cost 1.4 us.)
  int64_t tiles = ceil_div<int64_t>((int64_t)a.r.max_pages * a.c.ps, PR_T);
  if (a.window)
    tiles = std::min(tiles, (a.window + 2 * A.R) / PR_T + 2 + std::min(tiles, ceil_div<int64_t>(a.sinks, PR_T)));
  A.split = 1;
  while (A.split < 8 && blocks * A.split * 2 <= sms && tiles >= 2 * PR_MIN_STEPS * A.split) A.split *= 2;
  if (a.c.D <= 64)
    return e4m3 ? launch_prompt_t<64, true>(A, blocks, s) : launch_prompt_t<64, false>(A, blocks, s);
  return e4m3 ? launch_prompt_t<128, true>(A, blocks, s) : launch_prompt_t<128, false>(A, blocks, s);
}

}  // namespace bwta
