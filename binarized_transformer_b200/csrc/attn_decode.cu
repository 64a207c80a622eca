// attn_decode.cu -- attention of one new token of each sequence over the paged
// key-value cache.
//
// For every query head, o = sum_j w_j v_j / sum_j w_j with w_j = 2^(x_j - m) and
// x_j = softmax_scale * log2(e) * (q . k_j). The keys and values are read once:
// m, l = sum w and the weighted sum of the values are running values, rescaled
// by 2^(m_old - m_new) when the maximum grows. Two halves of the keys joined:
// m = max(m_a, m_b), l = l_a 2^(m_a - m) + l_b 2^(m_b - m), the same for the sums.
//
// Work: an item is a sequence's key head with up to 16 of its query heads, its
// units are the tiles of 64 tokens that hold a visible key. All units of the
// call in a row are cut into equal pieces, one for each block, so that lengths
// of any mix load the GPU evenly and one long sequence is spread over all of
// it. A block that covers an item alone writes the output; pieces of an item go
// to the workspace (at most two of a block: one item that began before it, one
// that goes on after it) and k_attn_join adds them in the order of the blocks, so
// the order of every sum is fixed by the lengths alone.
//
// Inside a block each of the 4 warps takes 16 tokens of a tile. page_size is a
// multiple of 16, so these lie in one page and are one contiguous piece of it.
// A warp copies its tokens into a ring of its own (cp.async, rows that are
// hidden or past the end are filled with zeros and never read) and needs no
// barrier but its own; the block meets only at the end of an item.
//
// The products run on mma.sync m16n8k16: the query heads of an item are the 16
// rows, which suits 1 .. 16 heads on one key head; the fifth-generation
// instructions would need 64 or 128 rows, and here HBM is the bound: per SM 23
// bytes a clock, i.e. one such instruction every 11 clocks of a pipe that takes one
// every 2. P is rounded to fp16 for the second product, l sums it unrounded.
// E4M3: K's scale is applied to the scores in fp32; V's, a power of two, to the
// converted values, which stays exact.
#include <algorithm>

#include "kv.cuh"
#include "tma.cuh"

namespace bwta {

constexpr int DEC_TILE = 64;     // tokens of a unit
constexpr int DEC_WARPS = 4, DEC_THREADS = DEC_WARPS * 32;
constexpr int DEC_SUB = DEC_TILE / DEC_WARPS;  // tokens of one warp in a unit
constexpr int DEC_ROWS = 16;     // query heads of an item
constexpr int DEC_MIN_UNITS = 1; // units that a block takes at least
constexpr int DEC_MAX_BLOCKS = 640;
constexpr int JOIN_THREADS = 256, JOIN_HEADS = JOIN_THREADS / 32;

template <int DP, bool E4M3>
struct DecShape {
  static constexpr int ROW = DP * (E4M3 ? 1 : 2);      // bytes of a token's row in the ring
  static constexpr int STAGES = E4M3 ? 6 : 3;
  static constexpr int HALF = DEC_SUB * ROW;           // keys (or values) of a stage
  static constexpr int STAGE = 2 * HALF + (E4M3 ? 2 * DEC_SUB * 4 : 0);
  static constexpr int RING = DEC_WARPS * STAGES * STAGE;
  static constexpr int PART = (DP / 2 + 4) * 32;       // floats of one warp's running values
  static constexpr int SMEM = RING + 2 * PART * 4;
  static_assert(2 * PART * 4 >= (DEC_THREADS + 1 + DEC_WARPS) * 8, "the prefix sums share the place");
};

struct DecArgs {
  AttnArgs a;
  float *ws;
  int groups;  // items of a key head: ceil(heads per key head / 16)
  int rows;    // heads of an item at most (rows of a piece in the workspace)
  int blocks;  // of k_attn_decode
};

// A sequence's tiles with a visible key: [0, sink_tiles) and [first, tiles).
struct DecSeq {
  int32_t slot, len, sink_tiles, first;
  int32_t units;
  bool bad;
};
__device__ __forceinline__ DecSeq dec_seq(const AttnArgs &a, int64_t s) {
  DecSeq q;
  q.bad = false;
  q.slot = kv_slot(a.r, s);
  q.len = kv_length(a.r, q.slot, a.c.ps, q.bad);
  const int32_t tiles = (q.len + DEC_TILE - 1) / DEC_TILE;
  q.sink_tiles = 0;
  q.first = 0;
  if (a.window && a.window < q.len) {
    q.first = (int32_t)((q.len - a.window) / DEC_TILE);
    q.sink_tiles = min((int32_t)((min(a.sinks, (int64_t)q.len) + DEC_TILE - 1) / DEC_TILE), q.first);
  }
  q.units = q.sink_tiles + tiles - q.first;
  return q;
}

// Units before each thread's share of the sequences (a share is `per` sequences),
// for blocks of T threads; before[T] = all of them.
template <int T>
__device__ __forceinline__ int dec_scan(const AttnArgs &a, int64_t *before, int64_t *sums) {
  const int per = (int)ceil_div<int64_t>(a.n_seq, T);
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int64_t s = (int64_t)threadIdx.x * per + i;
    if (s < a.n_seq) mine += dec_seq(a, s).units;
  }
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t x = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t y = __shfl_up_sync(FULL, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) base += sums[w];
    total += sums[w];
  }
  before[threadIdx.x] = base + x - mine;
  if (threadIdx.x == 0) before[T] = total;
  __syncthreads();
  return per;
}

// How the units are cut: block c has [start(c), start(c + 1)).
struct DecCut {
  int64_t total;
  int blocks;
  __device__ DecCut(int64_t t, int most) : total(t) {
    blocks = (int)min((int64_t)most, (t + DEC_MIN_UNITS - 1) / DEC_MIN_UNITS);
  }
  __device__ int64_t start(int c) const { return total * c / blocks; }
  __device__ int owner(int64_t u) const { return (int)(((u + 1) * blocks - 1) / total); }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool read) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
               "r"(read ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 bytes as two halves.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// Byte offset of 16-byte chunk c of row r: rows of 64, 128 or 256 bytes, chunks
// swizzled so that the 8 rows of one ldmatrix matrix fall on different banks.
template <int ROW>
__device__ __forceinline__ uint32_t ring_at(int r, int c) {
  return (uint32_t)(r * ROW + ((c ^ (ROW == 64 ? (r >> 1) & 3 : r & 7)) << 4));
}

// A position in a block's units: sequence, item, tile.
struct DecCursor {
  int64_t s;
  DecSeq q;
  int item, unit;  // item of the sequence, unit of the item
  __device__ void enter(const AttnArgs &a) {  // the first sequence with units from s on
    while (q.units == 0) q = dec_seq(a, ++s);
  }
  __device__ int tile() const { return unit < q.sink_tiles ? unit : q.first + unit - q.sink_tiles; }
};

template <int DP, bool E4M3>
__global__ void __launch_bounds__(DEC_THREADS, 2) k_attn_decode(const DecArgs A) {
  using S = DecShape<DP, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs &a = A.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int D = a.c.D, heads = a.n_heads / a.c.H, items = a.c.H * A.groups;
  const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
  float *joint = reinterpret_cast<float *>(smem + S::RING);
  int64_t *before = reinterpret_cast<int64_t *>(joint), *sums = before + DEC_THREADS + 1;

  pdl_trigger();
  if (D < DP)  // columns past D are never written: zero once
    for (int i = threadIdx.x * 16; i < S::RING; i += DEC_THREADS * 16)
      *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0, 0, 0, 0);
  pdl_wait();
  const int per = dec_scan<DEC_THREADS>(a, before, sums);  // its barriers cover the zeros
  const DecCut cut(before[DEC_THREADS] * items, A.blocks);
  if ((int)blockIdx.x >= cut.blocks) return;
  const int64_t u0 = cut.start(blockIdx.x), u1 = cut.start(blockIdx.x + 1);
  const int n = (int)(u1 - u0);
  if (n == 0) return;

  // the sequence, item and tile of unit u0
  DecCursor at;
  {
    int lo = 0, hi = DEC_THREADS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] * items <= u0) lo = mid;
      else hi = mid - 1;
    }
    int64_t u = u0 - before[lo] * items;
    at.s = (int64_t)lo * per;
    at.q = dec_seq(a, at.s);
    while (u >= (int64_t)at.q.units * items) {
      u -= (int64_t)at.q.units * items;
      at.q = dec_seq(a, ++at.s);
    }
    at.item = (int)(u / at.q.units);
    at.unit = (int)(u - (int64_t)at.item * at.q.units);
  }
  __syncthreads();  // the prefix sums have been read: `joint` may be written
  DecCursor ld = at;  // runs ahead of `at`: the copies
  int loaded = 0;
  bool bad = false, finite = true;

  // page of ld's tokens, fetched one unit before it is used
  auto page_of = [&](const DecCursor &c) -> int32_t {
    const int64_t tok = (int64_t)c.tile() * DEC_TILE + warp * DEC_SUB;
    return tok < c.q.len ? a.r.pages[(int64_t)c.q.slot * a.r.ld + tok / a.c.ps] : -1;
  };
  auto step = [&](DecCursor &c) {
    if (++c.unit < c.q.units) return;
    c.unit = 0;
    if (++c.item < items) return;
    c.item = 0;
    c.q = dec_seq(a, ++c.s);
    c.enter(a);
  };
  int32_t page = page_of(ld);
  auto load = [&]() {
    if (loaded < n) {
      const int tok = ld.tile() * DEC_TILE + warp * DEC_SUB, kh = ld.item / A.groups;
      const int rows = min(DEC_SUB, ld.q.len - tok);
      if (rows > 0) {
        const bool ok = (uint32_t)page < (uint32_t)a.c.num_pages;
        bad |= !ok;
        const int64_t row = (int64_t)kh * a.c.ps + tok % a.c.ps;
        const int64_t elt = (int64_t)(ok ? page : 0) * a.c.page_stride + row * D;
        const uint8_t *k = a.c.k + (E4M3 ? elt : 2 * elt), *v = a.c.v + (E4M3 ? elt : 2 * elt);
        const uint32_t st = ring + (loaded % S::STAGES) * S::STAGE;
        // visible rows of the 16: below `rows`, and not between the sinks and the window
        const int gap0 = a.window ? (int)min(max(a.sinks - tok, (int64_t)0), (int64_t)DEC_SUB) : DEC_SUB;
        const int gap1 = a.window ? (int)min(max(ld.q.len - a.window - tok, (int64_t)0), (int64_t)DEC_SUB) : 0;
        auto seen = [&](int r) { return ok && r < rows && (r < gap0 || r >= gap1); };
        const int width = D * (E4M3 ? 1 : 2);
        if (!E4M3 || D % 16 == 0) {
          const int chunks = width / 16;
          if (chunks == S::ROW / 16) {
#pragma unroll
            for (int i = 0; i < S::HALF / 512; ++i) {
              const int p = i * 32 + lane, r = p / (S::ROW / 16), c = p % (S::ROW / 16);
              cp_async16(st + ring_at<S::ROW>(r, c), k + p * 16, seen(r));
            }
#pragma unroll
            for (int i = 0; i < S::HALF / 512; ++i) {
              const int p = i * 32 + lane, r = p / (S::ROW / 16), c = p % (S::ROW / 16);
              cp_async16(st + S::HALF + ring_at<S::ROW>(r, c), v + p * 16, seen(r));
            }
          } else {
            for (int p = lane; p < DEC_SUB * chunks; p += 32) {
              const int r = p / chunks, c = p - r * chunks;
              const uint32_t to = st + ring_at<S::ROW>(r, c);
              cp_async16(to, k + p * 16, seen(r));
              cp_async16(to + S::HALF, v + p * 16, seen(r));
            }
          }
        } else {  // rows of 8 bytes more than a multiple of 16
          const int pieces = width / 8;
          for (int p = lane; p < DEC_SUB * pieces; p += 32) {
            const int r = p / pieces, c = p - r * pieces;
            const uint32_t to = st + ring_at<S::ROW>(r, c / 2) + (c & 1) * 8;
            cp_async8(to, k + p * 8, seen(r));
            cp_async8(to + S::HALF, v + p * 8, seen(r));
          }
        }
        if (E4M3 && lane < 8) {  // the rows' scales: 4 x 16 bytes of k, then of v
          const int c = lane % 4;
          const float *src = (lane < 4 ? a.c.ks : a.c.vs) + (int64_t)(ok ? page : 0) * a.c.scale_stride + row;
          cp_async16(st + 2 * S::HALF + lane * 16, src + c * 4, ok && c * 4 < rows);
        }
      }
      if (++loaded < n) {
        step(ld);
        page = page_of(ld);
      }
    }
    cp_commit();
  };

#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) load();

  constexpr int KS = DP / 16;
  uint32_t qa[KS][4];
  float o[DP / 8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  const float c2 = a.scale * 1.44269504088896340736f;
  bool fresh = true;
  for (int i = 0; i < n; ++i) {
    const int kh = at.item / A.groups, h0 = (at.item % A.groups) * DEC_ROWS;
    const int mine = min(DEC_ROWS, heads - h0);  // heads of this item
    if (fresh) {
      fresh = false;
      const uint16_t *q = a.q + at.s * a.ldq + (int64_t)(kh * heads + h0) * D;
      // fp16: k slots 2t, 2t+1 (and +8) of a step of 16 are those columns; E4M3: a
      // lane's four bytes of K are columns 4t .. 4t+3, so Q follows that order
      auto two = [&](int r, int d) -> uint32_t {
        return r < mine && d < D ? *reinterpret_cast<const uint32_t *>(q + (int64_t)r * D + d) : 0u;
      };
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int d0 = ks * 16 + (E4M3 ? 4 * t : 2 * t), d1 = d0 + (E4M3 ? 2 : 8);
        qa[ks][0] = two(g, d0);
        qa[ks][1] = two(g + 8, d0);
        qa[ks][2] = two(g, d1);
        qa[ks][3] = two(g + 8, d1);
      }
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
    }
    load();
    cp_wait<S::STAGES - 1>();
    __syncwarp();
    const int tok = at.tile() * DEC_TILE + warp * DEC_SUB;
    bad |= at.q.bad;
    if (tok < at.q.len) {
      const uint32_t st = ring + (i % S::STAGES) * S::STAGE;
      float s0[4] = {0, 0, 0, 0}, s1[4] = {0, 0, 0, 0};
      uint32_t r[4];
      const int mat = lane / 8, mr = lane % 8;
      if (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          ldsm4(st + ring_at<S::ROW>((mat / 2) * 8 + mr, ks * 2 + (mat & 1)), r);
          mma16816(s0, qa[ks], r[0], r[1]);
          mma16816(s1, qa[ks], r[2], r[3]);
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          ldsm4(st + ring_at<S::ROW>((mat & 1) * 8 + mr, ks + mat / 2), r);
          mma16816(s0, qa[ks], e4m3x2_to_half2(r[0]), e4m3x2_to_half2(r[0] >> 16));
          mma16816(s1, qa[ks], e4m3x2_to_half2(r[1]), e4m3x2_to_half2(r[1] >> 16));
          mma16816(s0, qa[ks + 1], e4m3x2_to_half2(r[2]), e4m3x2_to_half2(r[2] >> 16));
          mma16816(s1, qa[ks + 1], e4m3x2_to_half2(r[3]), e4m3x2_to_half2(r[3] >> 16));
        }
      }
      // scores: columns 2t, 2t+1 of s0 are tokens tok + 2t .., of s1 tok + 8 + 2t ..
      float f[4] = {c2, c2, c2, c2};
      const int64_t lo = a.window ? at.q.len - a.window : 0;
      bool vis[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = tok + (e / 2) * 8 + 2 * t + (e & 1);
        vis[e] = j < at.q.len && (j >= lo || j < a.sinks);
      }
      uint32_t vs01 = 0, vs23 = 0;
      if (E4M3) {
        const float2 *sc = reinterpret_cast<const float2 *>(smem + (st - smem_addr(smem)) + 2 * S::HALF);
        const float2 ka = sc[t], kb = sc[t + 4], va = sc[8 + t], vb = sc[12 + t];
        f[0] *= ka.x;
        f[1] *= ka.y;
        f[2] *= kb.x;
        f[3] *= kb.y;
        // a hidden token's scale may be anything, and its weight of 0 would not undo a NaN
        vs01 = half2_bits(vis[0] ? va.x : 0.0f, vis[1] ? va.y : 0.0f);
        vs23 = half2_bits(vis[2] ? vb.x : 0.0f, vis[3] ? vb.y : 0.0f);
      }
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[0][e] = vis[e] ? (e < 2 ? s0[e] : s1[e - 2]) * f[e] : -INFINITY;
        x[1][e] = vis[e] ? (e < 2 ? s0[e + 2] : s1[e]) * f[e] : -INFINITY;
      }
      float n0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3]));
      float n1 = fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        n0 = fmaxf(n0, __shfl_xor_sync(FULL, n0, d));
        n1 = fmaxf(n1, __shfl_xor_sync(FULL, n1, d));
      }
      n0 = fmaxf(n0, m0);
      n1 = fmaxf(n1, m1);
      if (__any_sync(FULL, n0 > m0 || n1 > m1)) {
        // nothing seen so far: the sums are zero and the factor does not matter
        const float a0 = m0 == -INFINITY ? 0.0f : exp2_fast(m0 - n0);
        const float a1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          o[j][0] *= a0;
          o[j][1] *= a0;
          o[j][2] *= a1;
          o[j][3] *= a1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
      float w[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[0][e] = exp2_fast(x[0][e] - z0);
        w[1][e] = exp2_fast(x[1][e] - z1);
      }
      l0 += (w[0][0] + w[0][1]) + (w[0][2] + w[0][3]);
      l1 += (w[1][0] + w[1][1]) + (w[1][2] + w[1][3]);
      const uint32_t pa[4] = {half2_bits(w[0][0], w[0][1]), half2_bits(w[1][0], w[1][1]),
                              half2_bits(w[0][2], w[0][3]), half2_bits(w[1][2], w[1][3])};
      if (!E4M3) {
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          ldsm4t(st + S::HALF + ring_at<S::ROW>((mat & 1) * 8 + mr, j * 2 + mat / 2), r);
          mma16816(o[2 * j], pa, r[0], r[1]);
          mma16816(o[2 * j + 1], pa, r[2], r[3]);
        }
      } else {
        // o[2j] holds the even columns of the j-th 16, o[2j + 1] the odd ones
#pragma unroll
        for (int j = 0; j < DP / 16; j += 2) {
          ldsm4t(st + S::HALF + ring_at<S::ROW>((mat & 1) * 8 + mr, j + mat / 2), r);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t a0 = r[2 * p], b0 = r[2 * p + 1];
            mma16816(o[2 * (j + p)], pa, mul_half2(e4m3x2_to_half2(__byte_perm(a0, 0, 0x20)), vs01),
                     mul_half2(e4m3x2_to_half2(__byte_perm(b0, 0, 0x20)), vs23));
            mma16816(o[2 * (j + p) + 1], pa, mul_half2(e4m3x2_to_half2(__byte_perm(a0, 0, 0x31)), vs01),
                     mul_half2(e4m3x2_to_half2(__byte_perm(b0, 0, 0x31)), vs23));
          }
        }
      }
    }
    __syncwarp();  // the stage may be filled again

    const bool item_ends = at.unit + 1 == at.q.units;
    if (item_ends || i == n - 1) {
      // join the warps: 1 into 0 and 3 into 2, then 2 into 0
      const int most = mine > 8 ? 4 : 2;  // rows g + 8 hold heads
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        l0 += __shfl_xor_sync(FULL, l0, d);
        l1 += __shfl_xor_sync(FULL, l1, d);
      }
      auto give = [&](float *p) {
        p[lane] = m0;
        p[32 + lane] = l0;
        p[64 + lane] = m1;
        p[96 + lane] = l1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < most)
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) p[(4 + e * (DP / 8) + j) * 32 + lane] = o[j][e];
      };
      auto join = [&](float &m, float &l, float pm, float pl, float &fa, float &fb) {
        const float M = fmaxf(m, pm);
        fa = m == -INFINITY ? 0.0f : exp2_fast(m - M);
        fb = pm == -INFINITY ? 0.0f : exp2_fast(pm - M);
        l = l * fa + pl * fb;
        m = M;
      };
      auto take = [&](const float *p) {
        float fa[2], fb[2];
        join(m0, l0, p[lane], p[32 + lane], fa[0], fb[0]);
        join(m1, l1, p[64 + lane], p[96 + lane], fa[1], fb[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < most)
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
              o[j][e] = o[j][e] * fa[e / 2] + p[(4 + e * (DP / 8) + j) * 32 + lane] * fb[e / 2];
      };
      if (warp & 1) give(joint + (warp / 2) * S::PART);
      __syncthreads();
      if (!(warp & 1)) take(joint + (warp / 2) * S::PART);
      if (warp == 2) give(joint + S::PART);
      __syncthreads();
      if (warp == 0) take(joint + S::PART);
      __syncthreads();
      if (warp == 0) {
        const bool began = i >= at.unit;  // the item's first unit is this block's too
        const bool whole = began && item_ends;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = g + 8 * half;
          if (row >= mine) continue;
          const float M = half ? m1 : m0, L = half ? l1 : l0;
          float *piece = A.ws + (((size_t)blockIdx.x * 2 + (began ? 1 : 0)) * A.rows + row) * (DP + 2);
          uint16_t *out = a.out + at.s * a.ldo + (int64_t)(kh * heads + h0 + row) * D;
          if (!whole && t == 0) *reinterpret_cast<float2 *>(piece + DP) = make_float2(M, L);
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            // E4M3: even columns in o[2i], odd ones in o[2i + 1]; two neighbours at once
            const int jj = E4M3 ? j & ~1 : j, e = E4M3 ? j & 1 : 0;
            const int col = E4M3 ? (j / 2) * 16 + 4 * t + 2 * e : j * 8 + 2 * t;
            float y0 = E4M3 ? o[jj][2 * half + e] : o[j][2 * half];
            float y1 = E4M3 ? o[jj + 1 < DP / 8 ? jj + 1 : jj][2 * half + e] : o[j][2 * half + 1];
            if (col >= D) continue;
            if (whole) {
              y0 /= L;
              y1 /= L;
              finite &= y0 - y0 == 0.0f && y1 - y1 == 0.0f;
              *reinterpret_cast<uint32_t *>(out + col) = half2_bits(y0, y1);
            } else {
              *reinterpret_cast<float2 *>(piece + col) = make_float2(y0, y1);
            }
          }
        }
      }
      fresh = true;
    }
    if (i + 1 < n) step(at);
  }
  cp_wait<0>();
  if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
  if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
}

// The outputs of items that several blocks share, and of empty sequences. A warp
// a query head, 4 columns a lane.
template <int DP>
__global__ void __launch_bounds__(JOIN_THREADS) k_attn_join(const DecArgs A) {
  __shared__ int64_t before[JOIN_THREADS + 1], sums[JOIN_THREADS / 32];
  const AttnArgs &a = A.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int hb = (a.n_heads + JOIN_HEADS - 1) / JOIN_HEADS;
  const int64_t s = blockIdx.x / hb;
  const int h = (int)(blockIdx.x - s * hb) * JOIN_HEADS + warp;
  const int D = a.c.D, heads = a.n_heads / a.c.H, items = a.c.H * A.groups;
  pdl_trigger();
  pdl_wait();
  const int per = dec_scan<JOIN_THREADS>(a, before, sums);
  if (h >= a.n_heads) return;
  const DecSeq q = dec_seq(a, s);
  uint16_t *out = a.out + s * a.ldo + (int64_t)h * D + lane * 4;
  if (q.units == 0) {
    if (q.bad && lane == 0 && h == 0) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
    if (lane * 4 < D) *reinterpret_cast<uint2 *>(out) = make_uint2(0, 0);
    return;
  }
  const DecCut cut(before[JOIN_THREADS] * items, A.blocks);
  const int who = (int)(s / per), kh = h / heads, hg = (h - kh * heads) / DEC_ROWS;
  int64_t u = before[who] * items;
  for (int64_t i = (int64_t)who * per; i < s; ++i) u += (int64_t)dec_seq(a, i).units * items;
  u += (int64_t)(kh * A.groups + hg) * q.units;
  const int first = cut.owner(u), last = cut.owner(u + q.units - 1);
  if (first == last) return;  // written by that block
  const int row = h - kh * heads - hg * DEC_ROWS;
  // a piece is its block's second one when the item begins in that block
  auto piece = [&](int c) {
    return A.ws + ((size_t)(c * 2 + (cut.start(c) <= u ? 1 : 0)) * A.rows + row) * (DP + 2);
  };
  float M = -INFINITY, L = 0.0f, y[4] = {0, 0, 0, 0};
  for (int c = first + lane; c <= last; c += 32) M = fmaxf(M, piece(c)[DP]);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(FULL, M, d));
#pragma unroll 4
  for (int c = first; c <= last; ++c) {
    const float *p = piece(c);
    const float f = p[DP] == -INFINITY ? 0.0f : exp2_fast(p[DP] - M);
    L += p[DP + 1] * f;
    if (lane * 4 < D) {
      const float2 v0 = *reinterpret_cast<const float2 *>(p + lane * 4);
      const float2 v1 = *reinterpret_cast<const float2 *>(p + lane * 4 + 2);
      y[0] += v0.x * f;
      y[1] += v0.y * f;
      y[2] += v1.x * f;
      y[3] += v1.y * f;
    }
  }
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] /= L;
    finite &= y[e] - y[e] == 0.0f;
  }
  if (lane * 4 < D) {
    *reinterpret_cast<uint2 *>(out) = make_uint2(half2_bits(y[0], y[1]), half2_bits(y[2], y[3]));
    if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
  }
}

int64_t attn_decode_ws(int64_t n_heads, int64_t n_kv_heads, int64_t head_dim) {
  const int64_t rows = std::min<int64_t>(n_heads / std::max<int64_t>(n_kv_heads, 1), DEC_ROWS);
  return (int64_t)DEC_MAX_BLOCKS * 2 * rows * ((head_dim <= 64 ? 64 : 128) + 2) * 4;
}

template <int DP, bool E4M3>
static cudaError_t launch_decode_t(DecArgs A, cudaStream_t s) {
  static SmemOptIn opt_in;
  auto kern = k_attn_decode<DP, E4M3>;
  constexpr int smem = DecShape<DP, E4M3>::SMEM;
  if (cudaError_t e = opt_in(kern, smem, true)) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  A.blocks = std::min(std::max(sms, 1) * 2, DEC_MAX_BLOCKS);
  if (cudaError_t e = launch_pdl(kern, dim3(A.blocks), dim3(DEC_THREADS), smem, s, A)) return e;
  const int64_t joins = A.a.n_seq * ceil_div<int64_t>(A.a.n_heads, JOIN_HEADS);
  return launch_pdl(k_attn_join<DP>, dim3((unsigned)joins), dim3(JOIN_THREADS), 0, s, A);
}

cudaError_t launch_attn_decode(const AttnArgs &a, bool e4m3, float *ws, cudaStream_t s) {
  DecArgs A = {};
  A.a = a;
  A.ws = ws;
  const int heads = a.n_heads / a.c.H;
  A.groups = (heads + DEC_ROWS - 1) / DEC_ROWS;
  A.rows = std::min(heads, DEC_ROWS);
  if (a.c.D <= 64) return e4m3 ? launch_decode_t<64, true>(A, s) : launch_decode_t<64, false>(A, s);
  return e4m3 ? launch_decode_t<128, true>(A, s) : launch_decode_t<128, false>(A, s);
}

}  // namespace bwta
