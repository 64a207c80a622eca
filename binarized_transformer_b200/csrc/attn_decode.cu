// attn_decode.cu -- attention of one new token of each sequence over the paged
// key-value cache.
//
// For every query head, o = sum_j w_j v_j / sum_j w_j with w_j = 2^(x_j - m) and
// x_j = softmax_scale * log2(e) * (q . k_j). The keys and values are read once:
// m (near the maximum of x), l = sum w and the weighted sum of the values are running
// values, rescaled by 2^(m_old - m_new) when m grows. Two halves of the keys joined:
// m = max(m_a, m_b), l = l_a 2^(m_a - m) + l_b 2^(m_b - m), the same for the sums.
//
// Work: an item is a sequence's key head with up to 16 of its query heads, its
// units are the tiles (64 tokens, E4M3 128) that hold a visible key. All units of
// the call in a row are cut into equal pieces, one for each block, so that lengths
// of any mix load the GPU evenly and one long sequence is spread over all of it. A
// block that covers an item alone writes the output; pieces of an item go to the
// workspace (at most two of a block: one item that began before it, one that goes
// on after it) and k_attn_join adds them in the order of the blocks, so the order
// of every sum is fixed by the lengths alone.
//
// Few items of no great length (CLUSTER) are the latency case: a cluster of 2 .. 8
// blocks takes an item, each an equal share of its tiles, and adds the parts up over
// distributed shared memory. No prefix sums, no second launch.
//
// Inside a block each of the 4 warps takes 16 (32) tokens of a tile. page_size is a
// multiple of 16, so 16 tokens lie in one page and are one contiguous piece of it.
// A warp copies its tokens into a ring of its own (cp.async, rows that are
// hidden or past the end are filled with zeros and never read) and needs no
// barrier but its own; the block meets only at the end of an item.
//
// The products run on mma.sync m16n8k16, transposed: 16 keys are the rows and 8
// query heads the columns (two such blocks for 9 .. 16 heads), then 16 columns of V
// the rows. So a key converted or loaded once meets all heads in one instruction and
// the running sums of 8 heads take 32 registers. The fifth-generation instructions
// would need 64 or 128 rows, and here HBM is the bound: 23 bytes a clock and SM.
//
// The reference m starts 7 below the maximum and follows it only when a score passes it
// by 15 (ATTN_HEAD, ATTN_SLACK): most tiles then need no maximum over the lanes. P is
// rounded to fp16 for the second product, l sums it unrounded. E4M3: K's scale is applied
// to the scores in fp32; V's, a power of two, to the converted values, which stays
// exact.
//
// Measured on a B200 (a copy moves 6.55 TB/s), call after call with inputs that change:
// fp16, 64 sequences of 0 .. 8191 tokens, 64 query heads on 8 key heads of 128: 1.29 GB in
// 212 us, 0.93 of the copy's rate; E4M3, 32 sequences, window 4096, 32 heads: 1.10 GB in
// 214 us, 0.78 (the same inputs again and again: 201 us); E4M3, one sequence of 250,001
// tokens: 0.53 GB in 101 us, 0.80. A longer cache costs 6.2 TB/s more, 0.94; the rest is
// the start, the ends of items and the last blocks (about 20 us). The arithmetic is
// hidden (without the second product the time is the same), the warps are not: two blocks
// an SM 236 us, 16-token steps 241. One token over 333 in fp16, in clusters: 7.4 us in a
// row, 10.3 alone: the launch and the chain length, page, keys, parts; in a table with
// room for 8192 tokens, which takes the other way, 11.2 and 13.4.
//
// Widths other than 64 and 128 copy piece by piece with divisions and a test of each row,
// and multiply over all of DP: bound by the issue slots, not by HBM. The ragged fp16 case
// at 112, 96, 80 and 40: 229, 212, 199 and 152 us (0.75, 0.70, 0.62, 0.40 of the copy's
// rate), the windowed E4M3 one 306, 278, 278 and 249 (0.48, 0.46, 0.38, 0.22).
#include <algorithm>

#include "kv.cuh"
#include "tma.cuh"

namespace bwta {

constexpr int DEC_WARPS = 4, DEC_THREADS = DEC_WARPS * 32;
constexpr int DEC_MAX_ROWS = 16;  // query heads of an item at most
constexpr int DEC_MAX_BLOCKS = 640;
constexpr int JOIN_THREADS = 256, JOIN_HEADS = JOIN_THREADS / 32;

__host__ __device__ constexpr int dec_tile(bool e4m3) { return e4m3 ? 128 : 64; }

template <int DP, bool E4M3, int NB>
struct DecShape {
  static constexpr int SUB = dec_tile(E4M3) / DEC_WARPS;  // tokens of one warp in a unit
  static constexpr int TILE = dec_tile(E4M3);
  static constexpr int ROW = DP * (E4M3 ? 1 : 2);      // bytes of a token's row in the ring
  static constexpr int BLOCKS = NB == 1 ? 3 : 2;  // on an SM; two for up to 8 heads: E4M3 244 us for 211
  static constexpr int STAGES = (NB == 1 ? 2 : 3) * (DP == 64 ? 2 : 1);
  static constexpr int HALF = SUB * ROW;               // keys (or values) of a stage
  static constexpr int STAGE = 2 * HALF + (E4M3 ? 2 * SUB * 4 : 0);
  static constexpr int RING = DEC_WARPS * STAGES * STAGE;
  static constexpr int PART = (DP / 16 * NB * 4 + 4 * NB) * 32;  // floats of one warp's running values
  static constexpr int SMEM = RING + PART * 4;
  static_assert(PART * 4 >= (DEC_THREADS + 1 + DEC_WARPS) * 8, "the prefix sums share the place");
  static_assert(BLOCKS * (SMEM + 1024) <= 233472, "shared memory of an SM");
};

struct DecArgs {
  AttnArgs a;
  float *ws;
  int groups;  // items of a key head
  int per_item;  // query heads of one: 8 or 16
  int rows;    // heads of an item at most (rows of a piece in the workspace)
  int blocks;  // of k_attn_decode
  int cluster; // blocks of an item (CLUSTER)
};

// Workspace: the pieces (two of a block), then k_attn_decode's prefix sums for the join.
__host__ __device__ constexpr int64_t dec_pieces(int rows, int DP) {
  return (int64_t)DEC_MAX_BLOCKS * 2 * rows * (DP + 2);  // floats; a multiple of 2
}
constexpr int DEC_PREFIX = DEC_THREADS + 1;  // 64-bit numbers

// A sequence's tiles with a visible key: [0, sink_tiles) and [first, tiles).
struct DecSeq {
  int32_t slot, len, sink_tiles, first;
  int32_t units;
  bool bad;
};
template <int TILE>
__device__ __forceinline__ DecSeq dec_seq(const AttnArgs &a, int64_t s) {
  DecSeq q;
  q.bad = false;
  q.slot = kv_slot(a.r, s);
  q.len = kv_length(a.r, q.slot, a.c.ps, q.bad);
  const int32_t tiles = (q.len + TILE - 1) / TILE;
  q.sink_tiles = 0;
  q.first = 0;
  if (a.window && a.window < q.len) {
    q.first = (int32_t)((q.len - a.window) / TILE);
    q.sink_tiles = min((int32_t)((min(a.sinks, (int64_t)q.len) + TILE - 1) / TILE), q.first);
  }
  q.units = q.sink_tiles + tiles - q.first;
  return q;
}

// Units before each thread's share of the sequences (a share is `per` sequences);
// before[T] = all of them.
template <int TILE>
__device__ __forceinline__ int dec_scan(const AttnArgs &a, int64_t *before, int64_t *sums) {
  constexpr int T = DEC_THREADS;
  const int per = (int)ceil_div<int64_t>(a.n_seq, T);
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int64_t s = (int64_t)threadIdx.x * per + i;
    if (s < a.n_seq) mine += dec_seq<TILE>(a, s).units;
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
    blocks = (int)min((int64_t)most, t);
  }
  __device__ int64_t start(int c) const { return div_pos(total * c, blocks); }
  __device__ int owner(int64_t u) const { return (int)div_pos((u + 1) * blocks - 1, total); }
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
// Four E4M3 bytes as two pairs of halves.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t four, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
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

// 8x8 halves, transposed among the lanes of a warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A position in a block's units: sequence, item, tile.
template <int TILE>
struct DecCursor {
  int64_t s;
  DecSeq q;
  int item, unit;  // item of the sequence, unit of the item
  __device__ void enter(const AttnArgs &a) {  // the first sequence with units from s on
    while (q.units == 0) q = dec_seq<TILE>(a, ++s);
  }
  __device__ int tile() const { return unit < q.sink_tiles ? unit : q.first + unit - q.sink_tiles; }
};

template <int DP, bool E4M3, int NB, bool CLUSTER>
__global__ void __launch_bounds__(DEC_THREADS, DecShape<DP, E4M3, NB>::BLOCKS) k_attn_decode(const DecArgs A) {
  using S = DecShape<DP, E4M3, NB>;
  constexpr int SUB = S::SUB, TILE = S::TILE, MT = SUB / 16, KS = DP / 16, ROWS = 8 * NB;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs &a = A.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int D = a.c.D, heads = a.n_heads / a.c.H, items = a.c.H * A.groups;
  const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
  float *joint = reinterpret_cast<float *>(smem + S::RING);
  int64_t *before = reinterpret_cast<int64_t *>(joint), *sums = before + DEC_THREADS + 1;

  if (D < DP)  // columns past D are never written: zero once
    for (int i = threadIdx.x * 16; i < S::RING; i += DEC_THREADS * 16)
      *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();
  DecCursor<TILE> at;
  int n = 0;
  if (CLUSTER) {
    const int id = blockIdx.x / A.cluster, rank = blockIdx.x - id * A.cluster;
    const int s = id / items;
    at.s = s;
    at.item = id - s * items;
    at.q = dec_seq<TILE>(a, s);
    at.unit = (int)div_pos((int64_t)at.q.units * rank, A.cluster);
    n = (int)div_pos((int64_t)at.q.units * (rank + 1), A.cluster) - at.unit;
  } else {
    const int per = dec_scan<TILE>(a, before, sums);
    const DecCut cut(before[DEC_THREADS] * items, A.blocks);
    if (blockIdx.x == 0) {  // what the join needs to find an item's pieces
      int64_t *prefix = reinterpret_cast<int64_t *>(A.ws + dec_pieces(A.rows, DP));
      for (int i = threadIdx.x; i < DEC_PREFIX; i += DEC_THREADS) prefix[i] = before[i];
    }
    if ((int)blockIdx.x >= cut.blocks) return;
    const int64_t u0 = cut.start(blockIdx.x);
    n = (int)(cut.start(blockIdx.x + 1) - u0);
    if (n == 0) return;
    // the sequence, item and tile of unit u0
    int lo = 0, hi = DEC_THREADS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] * items <= u0) lo = mid;
      else hi = mid - 1;
    }
    int64_t u = u0 - before[lo] * items;
    at.s = (int64_t)lo * per;
    at.q = dec_seq<TILE>(a, at.s);
    while (u >= (int64_t)at.q.units * items) {
      u -= (int64_t)at.q.units * items;
      at.q = dec_seq<TILE>(a, ++at.s);
    }
    at.item = (int)div_pos(u, at.q.units);
    at.unit = (int)(u - (int64_t)at.item * at.q.units);
  }
  __syncthreads();  // the zeros are there, the prefix sums have been read: `joint` may be written
  bool bad = false, finite = true;

  // ---- the copies run ahead: their own position, with the entry of the row of pages
  // (idx) and the token in that page (in) that this warp's first token falls on
  DecCursor<TILE> ld = at;
  int loaded = 0, idx = 0, in = 0;
  const int step_idx = TILE / a.c.ps, step_in = TILE - step_idx * a.c.ps;
  int32_t page[MT];  // fetched one unit before they are used
  auto first_token = [&](const DecCursor<TILE> &c) { return c.tile() * TILE + warp * SUB; };
  auto locate = [&]() {
    const int tok = first_token(ld);
    idx = tok / a.c.ps;
    in = tok - idx * a.c.ps;
  };
  auto fetch_pages = [&]() {
    const int tok = first_token(ld);
    const int32_t *row = a.r.pages + (int64_t)ld.q.slot * a.r.ld + idx;
#pragma unroll
    for (int h = 0; h < MT; ++h)
      page[h] = tok + 16 * h < ld.q.len ? row[h && in + 16 >= a.c.ps ? 1 : 0] : -1;
  };
  auto step = [&](DecCursor<TILE> &c) -> bool {  // true: not simply the next tile
    if (++c.unit < c.q.units) return c.unit == c.q.sink_tiles;
    c.unit = 0;
    if (++c.item < items) return true;
    c.item = 0;
    c.q = dec_seq<TILE>(a, ++c.s);
    c.enter(a);
    return true;
  };
  // which chunks of a 512-byte stretch this lane copies, and where they land
  constexpr int CH = S::ROW / 16, RPI = 32 / CH;  // chunks of a row, rows a copy of the warp covers
  auto load = [&]() {
    if (loaded < n) {
      const int tok = first_token(ld), kh = ld.item / A.groups;
      const uint32_t st = ring + (loaded % S::STAGES) * S::STAGE;
      const bool plain = tok + SUB <= ld.q.len &&
                         (!a.window || tok >= ld.q.len - a.window || tok + SUB <= a.sinks);
#pragma unroll
      for (int h = 0; h < MT; ++h) {
        const int tk = tok + 16 * h, rows = min(16, ld.q.len - tk);
        if (rows <= 0) break;
        const int inp = h && in + 16 >= a.c.ps ? 0 : in + 16 * h;
        const bool ok = (uint32_t)page[h] < (uint32_t)a.c.num_pages;
        bad |= !ok;
        const int64_t row = (int64_t)kh * a.c.ps + inp;
        const int64_t elt = (int64_t)(ok ? page[h] : 0) * a.c.page_stride + row * D;
        const uint8_t *k = a.c.k + (E4M3 ? elt : 2 * elt), *v = a.c.v + (E4M3 ? elt : 2 * elt);
        const uint32_t to = st + h * 16 * S::ROW;
        if (plain && ok && D == DP) {
#pragma unroll
          for (int i = 0; i < 16 / RPI; ++i)
            cp_async16(to + ring_at<S::ROW>(i * RPI + lane / CH, lane % CH), k + (i * 32 + lane) * 16, true);
#pragma unroll
          for (int i = 0; i < 16 / RPI; ++i)
            cp_async16(to + S::HALF + ring_at<S::ROW>(i * RPI + lane / CH, lane % CH), v + (i * 32 + lane) * 16, true);
        } else {
          // visible rows of the 16: below `rows`, and not between the sinks and the window
          const int gap0 = a.window ? (int)min(max(a.sinks - tk, (int64_t)0), (int64_t)16) : 16;
          const int gap1 = a.window ? (int)min(max(ld.q.len - a.window - tk, (int64_t)0), (int64_t)16) : 0;
          auto seen = [&](int r) { return ok && r < rows && (r < gap0 || r >= gap1); };
          const int width = D * (E4M3 ? 1 : 2);
          if (!E4M3 || D % 16 == 0) {
            const int chunks = width / 16;
            for (int p = lane; p < 16 * chunks; p += 32) {
              const int r = p / chunks, c = p - r * chunks;
              const uint32_t at16 = to + ring_at<S::ROW>(r, c);
              cp_async16(at16, k + p * 16, seen(r));
              cp_async16(at16 + S::HALF, v + p * 16, seen(r));
            }
          } else {  // rows of 8 bytes more than a multiple of 16
            const int pieces = width / 8;
            for (int p = lane; p < 16 * pieces; p += 32) {
              const int r = p / pieces, c = p - r * pieces;
              const uint32_t at8 = to + ring_at<S::ROW>(r, c / 2) + (c & 1) * 8;
              cp_async8(at8, k + p * 8, seen(r));
              cp_async8(at8 + S::HALF, v + p * 8, seen(r));
            }
          }
        }
        if (E4M3 && lane < 8) {  // the rows' scales: SUB of k, then of v
          const int c = lane % 4;
          const float *src = (lane < 4 ? a.c.ks : a.c.vs) + (int64_t)(ok ? page[h] : 0) * a.c.scale_stride + row;
          cp_async16(st + 2 * S::HALF + ((lane / 4) * SUB + h * 16 + c * 4) * 4, src + c * 4, ok && c * 4 < rows);
        }
      }
      if (++loaded < n) {
        if (step(ld)) {
          locate();
        } else {
          idx += step_idx;
          in += step_in;
          if (in >= a.c.ps) {
            in -= a.c.ps;
            ++idx;
          }
        }
        fetch_pages();
      }
    }
    cp_commit();
  };
  locate();
  fetch_pages();
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) load();

  // ---- the running values: columns of the tiles are heads 8 b + 2 t, + 1
  uint32_t qb[NB][KS][2];
  float o[NB][KS][4], m[NB][2], l[NB][2];
  const float c2 = a.scale * 1.44269504088896340736f;
  const int mat = lane / 8, mr = lane % 8;
  bool fresh = true;
  int stage = 0;
  for (int i = 0; i < n; ++i) {
    const int kh = at.item / A.groups, h0 = (at.item - kh * A.groups) * ROWS;
    const int mine = min(ROWS, heads - h0);  // heads of this item
    if (fresh) {
      fresh = false;
      const uint16_t *q = a.q + at.s * a.ldq + (int64_t)(kh * heads + h0) * D;
      // fp16: k slots 2t, 2t+1 (and +8) of a step of 16 are those columns; E4M3: a
      // lane's four bytes of K are columns 4t .. 4t+3, so Q follows that order
      auto two = [&](int r, int d) -> uint32_t {
        return r < mine && d < D ? *reinterpret_cast<const uint32_t *>(q + (int64_t)r * D + d) : 0u;
      };
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d0 = ks * 16 + (E4M3 ? 4 * t : 2 * t), d1 = d0 + (E4M3 ? 2 : 8);
          qb[b][ks][0] = two(8 * b + g, d0);
          qb[b][ks][1] = two(8 * b + g, d1);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[b][ks][e] = 0.0f;
        }
        m[b][0] = m[b][1] = -INFINITY;
        l[b][0] = l[b][1] = 0.0f;
      }
    }
    load();
    cp_wait<S::STAGES - 1>();
    __syncwarp();
    const int tok = first_token(at);
    bad |= at.q.bad;
    if (tok < at.q.len) {
      const uint32_t st = ring + stage * S::STAGE;
      float s[MT][NB][4];
#pragma unroll
      for (int h = 0; h < MT; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][b][e] = 0.0f;
      uint32_t r[4];
#pragma unroll
      for (int h = 0; h < MT; ++h) {
        if (!E4M3) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            ldsm4(st + ring_at<S::ROW>(h * 16 + (mat & 1) * 8 + mr, ks * 2 + mat / 2), r);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(s[h][b], r, qb[b][ks][0], qb[b][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            ldsm4(st + ring_at<S::ROW>(h * 16 + (mat & 1) * 8 + mr, ks + mat / 2), r);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              uint32_t ka[4];
              e4m3x4_to_half2(r[2 * p], ka[0], ka[2]);
              e4m3x4_to_half2(r[2 * p + 1], ka[1], ka[3]);
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816(s[h][b], ka, qb[b][ks + p][0], qb[b][ks + p][1]);
            }
          }
        }
      }
      // scores: rows g and g + 8 of each 16 tokens, columns 2t, 2t + 1
      const float *scales = reinterpret_cast<const float *>(smem + (st - smem_addr(smem)) + 2 * S::HALF);
#pragma unroll
      for (int h = 0; h < MT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = E4M3 ? c2 * scales[h * 16 + e * 8 + g] : c2;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            s[h][b][2 * e] *= f;
            s[h][b][2 * e + 1] *= f;
          }
        }
      const bool plain = tok + SUB <= at.q.len &&
                         (!a.window || tok >= at.q.len - a.window || tok + SUB <= a.sinks);
      if (!plain) {
        const int64_t lo = a.window ? at.q.len - a.window : 0;
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = tok + h * 16 + e * 8 + g;
            if (!(j < at.q.len && (j >= lo || j < a.sinks)))
#pragma unroll
              for (int b = 0; b < NB; ++b) s[h][b][2 * e] = s[h][b][2 * e + 1] = -INFINITY;
          }
      }
      bool up = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[0][b][e], s[0][b][2 + e]);
          if (MT == 2) x = fmaxf(fmaxf(x, s[MT - 1][b][e]), s[MT - 1][b][2 + e]);
          up |= x - m[b][e] > ATTN_SLACK;  // also from -infinity; m + slack could be rounded up to x
        }
      if (__any_sync(FULL, up)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[0][b][e], s[0][b][2 + e]);
            if (MT == 2) x = fmaxf(fmaxf(x, s[MT - 1][b][e]), s[MT - 1][b][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(FULL, x, d));
            const float mn = fmaxf(m[b][e], x - ATTN_HEAD);
            // nothing seen so far: the sums are zero and the factor does not matter
            const float f = m[b][e] == -INFINITY ? 0.0f : exp2_fast(m[b][e] - mn);
            m[b][e] = mn;
            l[b][e] *= f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              o[b][ks][e] *= f;
              o[b][ks][2 + e] *= f;
            }
          }
      }
      uint32_t pb[MT][NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float z0 = m[b][0] == -INFINITY ? 0.0f : m[b][0], z1 = m[b][1] == -INFINITY ? 0.0f : m[b][1];
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w0 = exp2_fast(s[h][b][2 * e] - z0), w1 = exp2_fast(s[h][b][2 * e + 1] - z1);
            l[b][0] += w0;
            l[b][1] += w1;
            pb[h][b][e] = transpose8(half2_bits(w0, w1));
          }
      }
#pragma unroll
      for (int h = 0; h < MT; ++h) {
        if (h > 0 && tok + 16 * h >= at.q.len) break;  // nothing was copied there
        if (!E4M3) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            ldsm4t(st + S::HALF + ring_at<S::ROW>(h * 16 + (mat / 2) * 8 + mr, ks * 2 + (mat & 1)), r);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(o[b][ks], r, pb[h][b][0], pb[h][b][1]);
          }
        } else {
          // rows g of a product are the even columns of 16, rows g + 8 the odd ones
          const float2 va = *reinterpret_cast<const float2 *>(scales + SUB + h * 16 + 2 * t);
          const float2 vb = *reinterpret_cast<const float2 *>(scales + SUB + h * 16 + 8 + 2 * t);
          uint32_t v01 = half2_bits(va.x, va.y), v23 = half2_bits(vb.x, vb.y);
          if (!plain) {
            // a hidden token's scale may be anything, and its weight of 0 would not undo a NaN
            const int64_t lo = a.window ? at.q.len - a.window : 0;
            auto vis = [&](int x) {
              const int j = tok + h * 16 + x;
              return j < at.q.len && (j >= lo || j < a.sinks);
            };
            v01 = half2_bits(vis(2 * t) ? va.x : 0.0f, vis(2 * t + 1) ? va.y : 0.0f);
            v23 = half2_bits(vis(8 + 2 * t) ? vb.x : 0.0f, vis(9 + 2 * t) ? vb.y : 0.0f);
          }
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            ldsm4t(st + S::HALF + ring_at<S::ROW>(h * 16 + (mat & 1) * 8 + mr, ks + mat / 2), r);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t x = r[2 * p], y = r[2 * p + 1];
              // bytes 0, 2 (the even column of two tokens) and 1, 3 (the odd one)
              uint32_t vv[4];
              e4m3x4_to_half2(__byte_perm(x, 0, 0x3120), vv[0], vv[1]);
              e4m3x4_to_half2(__byte_perm(y, 0, 0x3120), vv[2], vv[3]);
              vv[0] = mul_half2(vv[0], v01);
              vv[1] = mul_half2(vv[1], v01);
              vv[2] = mul_half2(vv[2], v23);
              vv[3] = mul_half2(vv[3], v23);
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816(o[b][ks + p], vv, pb[h][b][0], pb[h][b][1]);
            }
          }
        }
      }
    }
    __syncwarp();  // the stage may be filled again
    if (++stage == S::STAGES) stage = 0;

    const bool item_ends = at.unit + 1 == at.q.units;
    if (item_ends || i == n - 1) {
      // join the warps: 1, 2 and 3 into 0
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[b][e] += __shfl_xor_sync(FULL, l[b][e], d);
      auto give = [&](float *p) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[(b * 4 + 2 * e) * 32 + lane] = m[b][e];
            p[(b * 4 + 2 * e + 1) * 32 + lane] = l[b][e];
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[(4 * NB + (b * KS + ks) * 4 + e) * 32 + lane] = o[b][ks][e];
        }
      };
      auto take = [&](const float *p) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float pm = p[(b * 4 + 2 * e) * 32 + lane], pl = p[(b * 4 + 2 * e + 1) * 32 + lane];
            const float M = fmaxf(m[b][e], pm);
            const float fa = m[b][e] == -INFINITY ? 0.0f : exp2_fast(m[b][e] - M);
            const float fb = pm == -INFINITY ? 0.0f : exp2_fast(pm - M);
            l[b][e] = l[b][e] * fa + pl * fb;
            m[b][e] = M;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int x = e; x < 4; x += 2)
                o[b][ks][x] = o[b][ks][x] * fa + p[(4 * NB + (b * KS + ks) * 4 + x) * 32 + lane] * fb;
          }
      };
#pragma unroll 1
      for (int x = 1; x < DEC_WARPS; ++x) {
        if (warp == x) give(joint);
        __syncthreads();
        if (warp == 0) take(joint);
        __syncthreads();
      }
      if (CLUSTER && warp == 0) {
        // this block's share, rows of DP sums, the maximum and the sum of weights
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float *row = joint + (8 * b + 2 * t + e) * (DP + 2);
            if (g == 0) *reinterpret_cast<float2 *>(row + DP) = make_float2(m[b][e], l[b][e]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const int c0 = ks * 16 + (E4M3 ? 2 * g : g), c1 = c0 + (E4M3 ? 1 : 8);
              row[c0] = o[b][ks][e];
              row[c1] = o[b][ks][2 + e];
            }
          }
      } else if (warp == 0) {
        const bool began = i >= at.unit;  // the item's first unit is this block's too
        const bool whole = began && item_ends;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * b + 2 * t + e;
            if (row >= mine) continue;
            float *piece = A.ws + (((size_t)blockIdx.x * 2 + (began ? 1 : 0)) * A.rows + row) * (DP + 2);
            uint16_t *out = a.out + at.s * a.ldo + (int64_t)(kh * heads + h0 + row) * D;
            if (!whole && g == 0) *reinterpret_cast<float2 *>(piece + DP) = make_float2(m[b][e], l[b][e]);
            const float inv = 1.0f / l[b][e];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const float y0 = o[b][ks][e], y1 = o[b][ks][2 + e];  // sums, and means of them
              const float z0 = mean_to_f16_range(y0 * inv), z1 = mean_to_f16_range(y1 * inv);
              const int c0 = ks * 16 + (E4M3 ? 2 * g : g), c1 = c0 + (E4M3 ? 1 : 8);
              if (E4M3) {  // two neighbours
                if (c0 >= D) continue;
                if (whole) *reinterpret_cast<uint32_t *>(out + c0) = half2_bits(z0, z1);
                else *reinterpret_cast<float2 *>(piece + c0) = make_float2(y0, y1);
                if (whole) finite &= z0 - z0 == 0.0f && z1 - z1 == 0.0f;
              } else {
                if (c0 < D) {
                  if (whole) out[c0] = __half_as_ushort(__float2half_rn(z0));
                  else piece[c0] = y0;
                  if (whole) finite &= z0 - z0 == 0.0f;
                }
                if (c1 < D) {
                  if (whole) out[c1] = __half_as_ushort(__float2half_rn(z1));
                  else piece[c1] = y1;
                  if (whole) finite &= z1 - z1 == 0.0f;
                }
              }
            }
          }
      }
      fresh = true;
    }
    if (i + 1 < n) step(at);
  }
  cp_wait<0>();
  if (CLUSTER) {
    if (n == 0 && threadIdx.x < ROWS)  // no tile: a sum that no weights have says so
      *reinterpret_cast<float2 *>(joint + threadIdx.x * (DP + 2) + DP) = make_float2(-INFINITY, -1.0f);
    __syncwarp();
    cluster_sync();
    // each block adds up some rows: a warp a row, 4 columns a lane
    const int rank = blockIdx.x % A.cluster, kh = at.item / A.groups, h0 = (at.item - kh * A.groups) * ROWS;
    const uint32_t part = smem_addr(joint);
    if (rank == 0 && threadIdx.x == 0) bad |= at.q.bad;
    for (int row = rank + warp * A.cluster; row < min(ROWS, heads - h0); row += DEC_WARPS * A.cluster) {
      float M = -INFINITY, L = 0.0f, y[4] = {0, 0, 0, 0};
      for (int k = 0; k < A.cluster; ++k) M = fmaxf(M, cluster_ld2(part + (row * (DP + 2) + DP) * 4, k).x);
      for (int k = 0; k < A.cluster; ++k) {
        const float2 ml = cluster_ld2(part + (row * (DP + 2) + DP) * 4, k);
        if (ml.y == -1.0f) continue;
        // no score above -infinity there: the sums are zeros, or the NaN that the output has to show
        const float f = ml.x == -INFINITY ? 0.0f : exp2_fast(ml.x - M);
        L += ml.y * f;
        if (lane * 4 < D) {
          const float2 v0 = cluster_ld2(part + (row * (DP + 2) + lane * 4) * 4, k);
          const float2 v1 = cluster_ld2(part + (row * (DP + 2) + lane * 4 + 2) * 4, k);
          y[0] += v0.x * f;
          y[1] += v0.y * f;
          y[2] += v1.x * f;
          y[3] += v1.y * f;
        }
      }
      if (lane * 4 < D) {
        const float inv = at.q.units ? 1.0f / L : 0.0f;  // an empty sequence: zeros
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = mean_to_f16_range(y[e] * inv);
          finite &= y[e] - y[e] == 0.0f;
        }
        *reinterpret_cast<uint2 *>(a.out + at.s * a.ldo + (int64_t)(kh * heads + h0 + row) * D + lane * 4) =
            make_uint2(half2_bits(y[0], y[1]), half2_bits(y[2], y[3]));
      }
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its part is read
  }
  if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
  if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
}

// The outputs of items that several blocks share, and of empty sequences: a warp a
// query head, 4 columns a lane. WIDE, for calls of few items, each spread over many
// blocks: a block a query head, its warps take the pieces in turn. Where an item's units
// lie comes from k_attn_decode's prefix sums (scanning the lengths in every block would
// be work of n_seq^2).
template <int DP, int TILE, bool WIDE>
__global__ void __launch_bounds__(JOIN_THREADS) k_attn_join(const DecArgs A) {
  __shared__ float part[WIDE ? JOIN_HEADS : 1][DP + 2];
  const AttnArgs &a = A.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int hb = WIDE ? a.n_heads : (a.n_heads + JOIN_HEADS - 1) / JOIN_HEADS;
  const int64_t s = blockIdx.x / hb;
  const int hx = (int)(blockIdx.x - s * hb), h = WIDE ? hx : hx * JOIN_HEADS + warp;
  const int D = a.c.D, heads = a.n_heads / a.c.H, items = a.c.H * A.groups;
  const int64_t *prefix = reinterpret_cast<const int64_t *>(A.ws + dec_pieces(A.rows, DP));
  const int per = (int)ceil_div<int64_t>(a.n_seq, DEC_THREADS), who = (int)div_pos(s, per);
  const int kh = h / heads, hg = (h - kh * heads) / A.per_item, row = h - kh * heads - hg * A.per_item;
  // No early trigger: blocks of the next kernel that wait here already would take the
  // places of this one's (64 ragged sequences, call after call: 237 us for 211).
  pdl_wait();
  if (h >= a.n_heads) return;
  int64_t u = prefix[who];
  const int64_t total = prefix[DEC_THREADS];
  const DecSeq q = dec_seq<TILE>(a, s);
  if (per > 1) {  // the sequences between the share's first and this one
    int64_t x = 0;
    for (int64_t i = (int64_t)who * per + lane; i < s; i += 32) x += dec_seq<TILE>(a, i).units;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(FULL, x, d);
    u += x;
  }
  uint16_t *out = a.out + s * a.ldo + (int64_t)h * D + lane * 4;
  if (q.units == 0) {
    if (WIDE && warp > 0) return;
    if (q.bad && lane == 0 && h == 0) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
    if (lane * 4 < D) *reinterpret_cast<uint2 *>(out) = make_uint2(0, 0);
    return;
  }
  const DecCut cut(total * items, A.blocks);
  u = u * items + (int64_t)(kh * A.groups + hg) * q.units;
  const int first = cut.owner(u), last = cut.owner(u + q.units - 1);
  if (first == last) return;  // written by that block
  // a piece is its block's second one where the item begins: in the first block
  auto piece = [&](int c) {
    return A.ws + ((size_t)(c * 2 + (c == first ? 1 : 0)) * A.rows + row) * (DP + 2);
  };
  constexpr int BY = WIDE ? JOIN_HEADS : 1;
  float M = -INFINITY, L = 0.0f, y[4] = {0, 0, 0, 0};
  const bool col = lane * 4 < D;
  for (int c0 = first + (WIDE ? warp : 0); c0 <= last; c0 += 32 * BY) {
    // 32 pieces: a lane holds one's maximum and sum
    const int c = c0 + lane * BY, n = min(32, (last - c0) / BY + 1);
    float pm = -INFINITY, pl = 0.0f;
    if (c <= last) {
      const float2 ml = *reinterpret_cast<const float2 *>(piece(c) + DP);
      pm = ml.x;
      pl = ml.y;
    }
    float top = pm;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
    const float mn = fmaxf(M, top);
    const float old = M == -INFINITY ? 0.0f : exp2_fast(M - mn);
    const float f = pm == -INFINITY ? 0.0f : exp2_fast(pm - mn);
    M = mn;
    L = L * old + pl * f;  // this lane's share
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= old;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float fi = __shfl_sync(FULL, f, i);
      const float *p = piece(c0 + i * BY);
      if (col) {
        const float2 v0 = *reinterpret_cast<const float2 *>(p + lane * 4);
        const float2 v1 = *reinterpret_cast<const float2 *>(p + lane * 4 + 2);
        y[0] += v0.x * fi;
        y[1] += v0.y * fi;
        y[2] += v1.x * fi;
        y[3] += v1.y * fi;
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) L += __shfl_xor_sync(FULL, L, d);
  if (WIDE) {
    if (lane == 0) {
      part[warp][DP] = M;
      part[warp][DP + 1] = L;
    }
    if (col)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][lane * 4 + e] = y[e];
    __syncthreads();
    if (warp > 0) return;
    for (int w = 0; w < JOIN_HEADS; ++w) M = fmaxf(M, part[w][DP]);
    L = y[0] = y[1] = y[2] = y[3] = 0.0f;
    for (int w = 0; w < JOIN_HEADS; ++w) {
      const float f = part[w][DP] == -INFINITY ? 0.0f : exp2_fast(part[w][DP] - M);
      L += part[w][DP + 1] * f;
      if (col)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += part[w][lane * 4 + e] * f;
    }
  }
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = mean_to_f16_range(y[e] / L);
    finite &= y[e] - y[e] == 0.0f;
  }
  if (col) {
    *reinterpret_cast<uint2 *>(out) = make_uint2(half2_bits(y[0], y[1]), half2_bits(y[2], y[3]));
    if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
  }
}

int64_t attn_decode_ws(int64_t n_heads, int64_t n_kv_heads, int64_t head_dim) {
  const int64_t rows = std::min<int64_t>(n_heads / std::max<int64_t>(n_kv_heads, 1), DEC_MAX_ROWS);
  return dec_pieces((int)rows, head_dim <= 64 ? 64 : 128) * 4 + DEC_PREFIX * 8;
}

template <int DP, bool E4M3, int NB>
static cudaError_t launch_decode_t(DecArgs A, cudaStream_t s) {
  using S = DecShape<DP, E4M3, NB>;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  A.blocks = std::min(std::max(sms, 1) * S::BLOCKS, DEC_MAX_BLOCKS);
  // Clusters where all items run at once and no block can get more than 8 tiles (measured: one
  // token over 333 13.4 -> 10.3 us; the other way spreads any length over the whole GPU).
  const AttnArgs &a = A.a;
  const int64_t items = a.n_seq * a.c.H * A.groups;
  int64_t tiles = ceil_div<int64_t>((int64_t)a.r.max_pages * a.c.ps, S::TILE);
  if (a.window)
    tiles = std::min(tiles, a.window / S::TILE + 2 + std::min(tiles, ceil_div<int64_t>(a.sinks, S::TILE)));
  for (A.cluster = 8; A.cluster >= 2; A.cluster /= 2) {
    if (items * A.cluster > A.blocks) continue;
    if (tiles > 8 * A.cluster) break;
    static SmemOptIn opt_in;
    auto kern = k_attn_decode<DP, E4M3, NB, true>;
    if (cudaError_t e = opt_in(kern, S::SMEM, true)) return e;
    return launch_pdl_cluster(kern, dim3((unsigned)(items * A.cluster)), (unsigned)A.cluster, dim3(DEC_THREADS),
                              S::SMEM, s, A);
  }
  static SmemOptIn opt_in;
  auto kern = k_attn_decode<DP, E4M3, NB, false>;
  if (cudaError_t e = opt_in(kern, S::SMEM, true)) return e;
  if (cudaError_t e = launch_pdl(kern, dim3(A.blocks), dim3(DEC_THREADS), S::SMEM, s, A)) return e;
  // An item of a call with few of them is cut into many pieces.
  const bool wide = items * 16 <= A.blocks;
  const int64_t joins = a.n_seq * (wide ? a.n_heads : ceil_div<int64_t>(a.n_heads, JOIN_HEADS));
  return launch_pdl(wide ? k_attn_join<DP, S::TILE, true> : k_attn_join<DP, S::TILE, false>,
                    dim3((unsigned)joins), dim3(JOIN_THREADS), 0, s, A);
}

template <int DP, bool E4M3>
static cudaError_t launch_decode_heads(DecArgs A, cudaStream_t s) {
  const int heads = A.a.n_heads / A.a.c.H;
  A.per_item = heads <= 8 ? 8 : 16;  // more than 16 query heads on a key head: it is read again
  A.groups = (heads + A.per_item - 1) / A.per_item;
  A.rows = std::min(heads, A.per_item);
  return heads <= 8 ? launch_decode_t<DP, E4M3, 1>(A, s) : launch_decode_t<DP, E4M3, 2>(A, s);
}

cudaError_t launch_attn_decode(const AttnArgs &a, bool e4m3, float *ws, cudaStream_t s) {
  DecArgs A = {};
  A.a = a;
  A.ws = ws;
  if (a.c.D <= 64) return e4m3 ? launch_decode_heads<64, true>(A, s) : launch_decode_heads<64, false>(A, s);
  return e4m3 ? launch_decode_heads<128, true>(A, s) : launch_decode_heads<128, false>(A, s);
}

}  // namespace bwta
