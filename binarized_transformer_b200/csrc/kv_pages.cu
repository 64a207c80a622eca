// kv_pages.cu -- the pages of the paged key-value cache: handed out to growing
// slots, given up, shared by forks, moved to the front of the pool, copied.
//
// The table lives on the device and so does every decision. One block plans a
// call: it turns the pool's counts into a bitmap of free pages in shared
// memory with a prefix of popcounts over it, so that "the r-th free page" is a
// search in shared memory, every request's pages are known from a prefix sum
// over the list, and the outcome does not depend on the order in which threads
// run. A second launch of many blocks then moves the pages' bytes (a copy,
// bound by HBM) and rewrites the rows. Plans read 4 bytes a page and a few a
// request: they are bound by latency.
//
// No pointer here is declared const __restrict__: a load through such a pointer
// may be moved above griddepcontrol.wait, and these kernels read what the kernel
// before them in the stream wrote.
#include <algorithm>

#include "kv.cuh"

namespace bwta {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_PER = BWTA_KV_MAX_LIST / PLAN_THREADS;  // list entries of one thread
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_PIECE = MOVE_THREADS * 16 * 4;  // bytes that one block copies at a time
constexpr int EDIT_CHUNK = 1024;                   // entries of a row edited by one block at a time

// Workspace, in int32: a header, then the list of copies, then what the rows need.
constexpr int WS_COUNT = 0, WS_USED = 1, WS_LIST = 16;

// ------------------------------------------------------------ the plan's tools
// Exclusive prefix sum over the block's threads; *total = the sum.
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(FULL, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the previous call's readers are done with warp_sums
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = lane < PLAN_THREADS / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(FULL, w, d);
    if (lane >= d) w += y;
  }
  *total = __shfl_sync(FULL, w, 31);
  const int before = __shfl_sync(FULL, w, (warp + 31) % 32);
  return x - v + (warp ? before : 0);
}

// The free pages of a pool as a bitmap (bit i of word w = page 32 w + i) with the
// number of free pages before each thread's share of the words.
struct FreeMap {
  uint32_t *bits;  // [words]
  int *before;     // [PLAN_THREADS + 1]
  int words, per;  // per = words of one thread
  int num, free;

  __device__ void build(const int32_t *ref, int num_pages, int *warp_sums) {
    num = num_pages;
    words = (num_pages + 31) / 32;
    per = (words + PLAN_THREADS - 1) / PLAN_THREADS;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    constexpr int U = 8;  // loads in flight
    for (int w0 = warp * U; w0 < words; w0 += PLAN_THREADS / 32 * U) {
      int r[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = (w0 + i) * 32 + lane;
        r[i] = p < num_pages ? ref[p] : 1;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t b = __ballot_sync(FULL, r[i] <= 0);
        if (lane == 0 && w0 + i < words) bits[w0 + i] = b;
      }
    }
    __syncthreads();
    int c = 0;
    for (int w = threadIdx.x * per; w < min(words, (int)(threadIdx.x + 1) * per); ++w)
      c += __popc(bits[w]);
    const int x = block_prefix(c, warp_sums, &free);
    before[threadIdx.x] = x;
    if (threadIdx.x == 0) before[PLAN_THREADS] = free;
    __syncthreads();
  }

  template <bool FREE>
  __device__ int count_before(int t) const {
    return FREE ? before[t] : min(t * per * 32, num) - before[t];
  }
  // The r-th free (or used) page, counted from 0; r is below their number.
  template <bool FREE>
  __device__ int select(int r) const {
    int lo = 0, hi = PLAN_THREADS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (count_before<FREE>(mid) <= r) lo = mid;
      else hi = mid - 1;
    }
    r -= count_before<FREE>(lo);
    for (int w = lo * per;; ++w) {
      uint32_t m = FREE ? bits[w] : ~bits[w];
      const int c = __popc(m);
      if (r < c) {
        for (; r > 0; --r) m &= m - 1;
        return w * 32 + __ffs(m) - 1;
      }
      r -= c;
    }
  }
};

// The first entry of a list with each value, by a table of twice its length in
// shared memory: after a barrier, owner(key, cell) tells whether entry i came
// first. Keys are >= 0.
struct FirstOf {
  int *key, *idx;
  int mask;

  __device__ void clear(int n) {
    int size = 2;
    while (size < 2 * n) size *= 2;
    mask = size - 1;
    for (int i = threadIdx.x; i < size; i += PLAN_THREADS) {
      key[i] = -1;
      idx[i] = 0x7fffffff;
    }
  }
  __device__ int insert(int k, int i) {
    uint32_t h = ((uint32_t)k * 2654435761u >> 7) & mask;
    for (;;) {  // at most half full: an empty cell or the key is found
      const int old = atomicCAS(&key[h], -1, k);
      if (old == -1 || old == k) break;
      h = (h + 1) & mask;
    }
    atomicMin(&idx[h], i);
    return (int)h;
  }
};

struct PlanSmem {
  int warp_sums[32];
  int before[PLAN_THREADS + 1];
  int need_before[BWTA_KV_MAX_LIST + 1];  // pages asked for by the requests before i
  int granted;
};
// dynamic shared memory: PlanSmem, hash keys and indices, bitmap
static size_t plan_smem(int64_t num_pages, int64_t n) {
  int64_t size = 2;
  while (size < 2 * n) size *= 2;
  return sizeof(PlanSmem) + (size_t)size * 8 + (size_t)((num_pages + 31) / 32) * 4 + 64;
}

// Hand out pages to the requests of a list: needs[] (this thread's PLAN_PER
// entries, entry i = threadIdx.x * PLAN_PER + j) -> which are met, and the prefix
// in sm->need_before for take().
__device__ __forceinline__ void plan_needs(PlanSmem *sm, const FreeMap &fm, int n,
                                           const int (&need)[PLAN_PER], bool (&met)[PLAN_PER]) {
  int mine = 0, total;
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) mine += need[j];
  if (threadIdx.x == 0) sm->granted = 0;
  int x = block_prefix(mine, sm->warp_sums, &total);
  int granted = 0;
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    if (i < n) sm->need_before[i] = x;
    x += need[j];
    met[j] = need[j] == 0 || x <= fm.free;
    if (x <= fm.free) granted = x;
  }
  if (threadIdx.x == 0) sm->need_before[n] = total;
  atomicMax(&sm->granted, granted);
  __syncthreads();
}

// The request that rank r (a page handed out) belongs to.
__device__ __forceinline__ int plan_owner(const PlanSmem *sm, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm->need_before[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Pages that a length takes; -1 for a length that the row cannot hold.
__device__ __forceinline__ int64_t pages_of(int64_t len, int ps, int max_pages) {
  if (len < 0) return -1;
  const int64_t p = (len + ps - 1) / ps;
  return p <= max_pages ? p : -1;
}

__device__ __forceinline__ void carve(uint8_t *raw, int64_t n, PlanSmem *&sm, FirstOf &first,
                                      FreeMap &fm) {
  sm = reinterpret_cast<PlanSmem *>(raw);
  int size = 2;
  while (size < 2 * n) size *= 2;
  first.key = reinterpret_cast<int *>(raw + sizeof(PlanSmem));
  first.idx = first.key + size;
  fm.bits = reinterpret_cast<uint32_t *>(first.idx + size);
  fm.before = sm->before;
}

// ------------------------------------------------------------------- reserve
__global__ void __launch_bounds__(PLAN_THREADS, 1)
k_kv_reserve(KvTableView t, int num_pages, int ps, const int32_t *slots,
             const int32_t *n_new, int n, int32_t *d_status) {
  extern __shared__ __align__(16) uint8_t raw[];
  PlanSmem *sm;
  FirstOf first;
  FreeMap fm;
  carve(raw, n, sm, first, fm);
  pdl_trigger();
  first.clear(n);
  pdl_wait();
  __syncthreads();

  int slot[PLAN_PER], cell[PLAN_PER], need[PLAN_PER];
  int64_t len[PLAN_PER];
  bool ok[PLAN_PER], met[PLAN_PER], bad = false, none = false;
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    slot[j] = i < n ? slots[i] : -1;
    ok[j] = (uint32_t)slot[j] < (uint32_t)t.n_slots;
    bad |= i < n && !ok[j];
    cell[j] = ok[j] ? first.insert(slot[j], i) : -1;
  }
  fm.build(t.ref, num_pages, sm->warp_sums);  // its barriers also settle the first entries
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    need[j] = 0;
    len[j] = 0;
    if (!ok[j]) continue;
    const int grow = n_new[i];
    const int64_t old = t.len[slot[j]];
    const int64_t h = pages_of(old, ps, t.max_pages);
    const int64_t w = grow < 0 || h < 0 ? -1 : pages_of(old + grow, ps, t.max_pages);
    ok[j] = first.idx[cell[j]] == i && w >= 0 && old + grow <= 0x7fffffff;
    bad |= !ok[j];
    if (!ok[j]) continue;
    need[j] = (int)min(w - h, (int64_t)num_pages + 1);  // more than the pool holds is never met
    len[j] = old + grow;
  }
  plan_needs(sm, fm, n, need, met);
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    if (!ok[j]) continue;
    none |= !met[j];
    if (met[j]) t.len[slot[j]] = (int32_t)len[j];
  }
  // Rank by rank. The request may be another thread's: its new entries are the
  // last ones of its row, whose length has been raised.
  __syncthreads();
  for (int r = threadIdx.x; r < sm->granted; r += PLAN_THREADS) {
    const int i = plan_owner(sm, n, r);
    const int s = slots[i];
    const int page = fm.select<true>(r);
    const int want = (int)pages_of(t.len[s], ps, t.max_pages);
    t.pages[(int64_t)s * t.ld + want - (sm->need_before[i + 1] - r)] = page;
    t.ref[page] = 1;
  }
  if (bad) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
  if (none) flag_status(d_status, BWTA_STATUS_NO_PAGE);
}

// ---------------------------------------------------------------------- fork
// The plan. Workspace: list of copies (cap entries each of source and target
// page, -1 = none), then 4 x n for the rows: source slot (-1 = fork not made), target
// slot, full pages, page of the unfilled rest (-1 = none).
__global__ void __launch_bounds__(PLAN_THREADS, 1)
k_kv_fork_plan(KvTableView t, int num_pages, int ps, const int32_t *src,
               const int32_t *dst, int n, int32_t *ws,
               int64_t cap, int32_t *d_status) {
  extern __shared__ __align__(16) uint8_t raw[];
  PlanSmem *sm;
  FirstOf first;
  FreeMap fm;
  carve(raw, n, sm, first, fm);
  pdl_trigger();
  first.clear(n);
  pdl_wait();
  __syncthreads();

  int from[PLAN_PER], to[PLAN_PER], cell[PLAN_PER], need[PLAN_PER], len[PLAN_PER];
  bool ok[PLAN_PER], met[PLAN_PER], bad = false, none = false;
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    from[j] = i < n ? src[i] : -1;
    to[j] = i < n ? dst[i] : -1;
    const bool to_ok = (uint32_t)to[j] < (uint32_t)t.n_slots;
    ok[j] = to_ok && (uint32_t)from[j] < (uint32_t)t.n_slots;
    bad |= i < n && !ok[j];
    cell[j] = to_ok ? first.insert(to[j], i) : -1;
  }
  fm.build(t.ref, num_pages, sm->warp_sums);
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    need[j] = 0;
    len[j] = 0;
    if (!ok[j]) continue;
    len[j] = t.len[from[j]];
    ok[j] = first.idx[cell[j]] == i && t.len[to[j]] == 0 && pages_of(len[j], ps, t.max_pages) >= 0;
    bad |= !ok[j];
    need[j] = ok[j] && len[j] % ps != 0;
  }
  plan_needs(sm, fm, n, need, met);  // every length has been read: they may change now
  int32_t *list_src = ws + WS_LIST, *list_dst = list_src + cap, *rows = list_dst + cap;
#pragma unroll
  for (int j = 0; j < PLAN_PER; ++j) {
    const int i = threadIdx.x * PLAN_PER + j;
    if (i >= n) continue;
    const bool made = ok[j] && met[j];
    none |= ok[j] && !met[j];
    int page = -1, old = -1;
    if (made && need[j]) {
      page = fm.select<true>(sm->need_before[i]);
      t.ref[page] = 1;
      old = t.pages[(int64_t)from[j] * t.ld + len[j] / ps];
    }
    const bool copy = page >= 0 && (uint32_t)old < (uint32_t)num_pages;
    bad |= page >= 0 && !copy;
    list_src[i] = copy ? old : -1;
    list_dst[i] = page;
    rows[4 * i + 0] = made ? from[j] : -1;
    rows[4 * i + 1] = to[j];
    rows[4 * i + 2] = len[j] / ps;
    rows[4 * i + 3] = page;
    if (made) t.len[to[j]] = len[j];
  }
  if (threadIdx.x == 0) ws[WS_COUNT] = n;
  if (bad) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
  if (none) flag_status(d_status, BWTA_STATUS_NO_PAGE);
}

// ------------------------------------------------------------------- compact
// The plan. Workspace: the list of moves, then the new number of each page that
// is not below the number in use ([num_pages], -1 for the free ones).
__global__ void __launch_bounds__(PLAN_THREADS, 1)
k_kv_compact_plan(KvTableView t, int num_pages, int32_t *n_used, int32_t *ws,
                  int64_t cap) {
  extern __shared__ __align__(16) uint8_t raw[];
  PlanSmem *sm;
  FirstOf first;
  FreeMap fm;
  carve(raw, 0, sm, first, fm);
  pdl_trigger();
  pdl_wait();
  fm.build(t.ref, num_pages, sm->warp_sums);
  const int used = num_pages - fm.free;
  // free pages below `used`: as many as used pages at or past it
  int c = 0, moves;
  for (int w = threadIdx.x; w * 32 < used; w += PLAN_THREADS) {
    const int left = used - w * 32;
    c += __popc(fm.bits[w] & (left >= 32 ? FULL : (1u << left) - 1));
  }
  block_prefix(c, sm->warp_sums, &moves);
  int32_t *list_src = ws + WS_LIST, *list_dst = list_src + cap, *map = list_dst + cap;
  for (int p = used + threadIdx.x; p < num_pages; p += PLAN_THREADS)
    if (fm.bits[p >> 5] >> (p & 31) & 1) map[p] = -1;
  for (int i = threadIdx.x; i < moves; i += PLAN_THREADS) {
    const int hole = fm.select<true>(i), far = fm.select<false>(used - moves + i);
    list_src[i] = far;
    list_dst[i] = hole;
    map[far] = hole;
    t.ref[hole] = t.ref[far];
    t.ref[far] = 0;
  }
  if (threadIdx.x == 0) {
    ws[WS_COUNT] = moves;
    ws[WS_USED] = used;
    if (n_used) *n_used = used;
  }
}

// ---------------------------------------------------------------------- copy
// The plan of bwta_kv_copy_pages: which copies of the list are made.
__global__ void __launch_bounds__(PLAN_THREADS, 1)
k_kv_copy_plan(int src_pages, int dst_pages, bool same, const int32_t *src,
               const int32_t *dst, int64_t n, int32_t *ws,
               int64_t cap, int32_t *d_status) {
  extern __shared__ __align__(16) uint32_t maps[];
  const int words = (dst_pages + 31) / 32;
  uint32_t *once = maps, *twice = maps + words;
  pdl_trigger();
  for (int w = threadIdx.x; w < 2 * words; w += PLAN_THREADS) maps[w] = 0;
  pdl_wait();
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += PLAN_THREADS) {
    const uint32_t d = (uint32_t)dst[i], s = (uint32_t)src[i], bit = 1u << (d & 31);
    if (d >= (uint32_t)dst_pages || s >= (uint32_t)src_pages) continue;
    if (atomicOr(&once[d >> 5], bit) & bit) atomicOr(&twice[d >> 5], bit);
  }
  __syncthreads();
  bool bad = false;
  for (int64_t i = threadIdx.x; i < n; i += PLAN_THREADS) {
    const uint32_t d = (uint32_t)dst[i], s = (uint32_t)src[i];
    bool ok = d < (uint32_t)dst_pages && s < (uint32_t)src_pages;
    ok = ok && !(twice[d >> 5] >> (d & 31) & 1);
    ok = ok && !(same && s != d && (once[s >> 5] >> (s & 31) & 1));
    bad |= !ok;
    ws[WS_LIST + i] = ok && !(same && s == d) ? (int32_t)s : -1;
    ws[WS_LIST + cap + i] = (int32_t)d;
  }
  if (threadIdx.x == 0) ws[WS_COUNT] = (int32_t)n;
  if (bad) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
}

// ---------------------------------------------------------------------- free
// One block a slot. The exchange of the length makes the first block that comes
// to a slot its only one.
__global__ void __launch_bounds__(256)
k_kv_free(KvTableView t, int num_pages, int ps, const int32_t *slots,
          int32_t *d_status) {
  __shared__ int s_len;
  pdl_trigger();
  pdl_wait();
  const int slot = slots[blockIdx.x];
  if ((uint32_t)slot >= (uint32_t)t.n_slots) {
    if (threadIdx.x == 0) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(&t.len[slot], 0);
  __syncthreads();
  const int64_t room = (int64_t)t.max_pages * ps;
  bool bad = s_len < 0 || s_len > room;
  const int n = (int)((min(max((int64_t)s_len, (int64_t)0), room) + ps - 1) / ps);
  int32_t *row = t.pages + (int64_t)slot * t.ld;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int p = row[i];
    row[i] = -1;
    if ((uint32_t)p >= (uint32_t)num_pages) {
      bad = true;
    } else if (atomicSub(&t.ref[p], 1) <= 0) {
      atomicAdd(&t.ref[p], 1);
      bad = true;
    }
  }
  if (bad) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
}

// ---------------------------------------------------------------------- move
enum { EDIT_NONE = 0, EDIT_FORK = 1, EDIT_COMPACT = 2 };

// 16-byte pieces of `bytes` bytes, by one block, four loads in flight a thread.
__device__ __forceinline__ void copy_piece(const uint8_t *src, uint8_t *dst, int64_t bytes) {
  const uint4 *s = reinterpret_cast<const uint4 *>(src);
  uint4 *d = reinterpret_cast<uint4 *>(dst);
  const int n = (int)(bytes / 16);
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = threadIdx.x + i * MOVE_THREADS;
    if (at < n) v[i] = __ldcs(s + at);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = threadIdx.x + i * MOVE_THREADS;
    if (at < n) __stcs(d + at, v[i]);
  }
}

// The copies of the plan's list in every layer, in pieces handed out round-robin,
// and the rows. Sources and targets of one list never overlap. `cap` is the
// capacity of the list (where its second half begins).
template <int EDIT>
__global__ void __launch_bounds__(MOVE_THREADS)
k_kv_move(const __grid_constant__ KvLayers l, const KvGeometry g, const KvTableView t,
          const int32_t *ws, int64_t cap, int32_t *d_status) {
  pdl_trigger();
  pdl_wait();
  const int64_t count = ws[WS_COUNT];
  const int kp = (int)ceil_div<int64_t>(g.kv_bytes, MOVE_PIECE);
  const int sp = (int)ceil_div<int64_t>(g.sc_bytes, MOVE_PIECE);
  const int64_t per_layer = 2 * (kp + sp), per_copy = per_layer * g.n_layers;
  for (int64_t task = blockIdx.x; task < count * per_copy; task += gridDim.x) {
    const int64_t c = task / per_copy;
    const int32_t from = ws[WS_LIST + c], to = ws[WS_LIST + cap + c];
    if (from < 0) continue;
    const int rest = (int)(task - c * per_copy), layer = rest / (int)per_layer;
    int piece = rest % (int)per_layer;
    const KvLayer &a = l.src[layer], &b = l.dst[layer];
    const bool second = piece >= kp + sp;  // k, then v
    if (second) piece -= kp + sp;
    if (piece < kp) {
      const int64_t off = (int64_t)piece * MOVE_PIECE;
      copy_piece((second ? a.v : a.k) + from * g.src_kv_stride + off,
                 (second ? b.v : b.k) + to * g.dst_kv_stride + off,
                 min((int64_t)MOVE_PIECE, g.kv_bytes - off));
    } else {
      const int64_t off = (int64_t)(piece - kp) * MOVE_PIECE;
      copy_piece(reinterpret_cast<const uint8_t *>(second ? a.vs : a.ks) + from * g.src_sc_stride + off,
                 reinterpret_cast<uint8_t *>(second ? b.vs : b.ks) + to * g.dst_sc_stride + off,
                 min((int64_t)MOVE_PIECE, g.sc_bytes - off));
    }
  }
  if (EDIT == EDIT_NONE) return;
  // rows, in chunks
  const int chunks = (int)ceil_div<int64_t>(t.max_pages, EDIT_CHUNK);
  const int64_t nrows = EDIT == EDIT_FORK ? count : t.n_slots;
  bool bad = false;
  for (int64_t task = blockIdx.x; task < nrows * chunks; task += gridDim.x) {
    const int64_t r = task / chunks;
    const int lo = (int)(task - r * chunks) * EDIT_CHUNK;
    if (EDIT == EDIT_FORK) {
      const int4 f = *reinterpret_cast<const int4 *>(ws + WS_LIST + 2 * cap + 4 * r);
      if (f.x < 0) continue;
      const int32_t *from = t.pages + (int64_t)f.x * t.ld;
      int32_t *to = t.pages + (int64_t)f.y * t.ld;
      for (int i = lo + threadIdx.x; i < min(lo + EDIT_CHUNK, f.z); i += MOVE_THREADS) {
        const int32_t p = from[i];
        to[i] = p;
        if ((uint32_t)p < (uint32_t)g.src_pages) atomicAdd(&t.ref[p], 1);
        else bad = true;
      }
      if (f.w >= 0 && threadIdx.x == 0 && f.z >= lo && f.z < lo + EDIT_CHUNK) to[f.z] = f.w;
    } else {
      const int64_t len = t.len[r];
      const int64_t own = min((max(len, (int64_t)0) + g.page_size - 1) / g.page_size, (int64_t)t.max_pages);
      bad |= len < 0 || len > (int64_t)t.max_pages * g.page_size;
      const int32_t used = ws[WS_USED];
      const int32_t *map = ws + WS_LIST + 2 * cap;
      int32_t *row = t.pages + r * t.ld;
      for (int i = lo + threadIdx.x; i < min((int64_t)lo + EDIT_CHUNK, own); i += MOVE_THREADS) {
        const int32_t p = row[i];
        // a page that a slot holds and nobody counts has no new number
        const int32_t to = (uint32_t)p >= (uint32_t)g.src_pages ? -1 : p < used ? p : map[p];
        if (to < 0) bad = true;
        else if (to != p) row[i] = to;
      }
    }
  }
  if (bad) flag_status(d_status, BWTA_STATUS_BAD_PAGE);
}

// ----------------------------------------------------------------- launchers
static int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::max(sms, 1);
}

static int64_t list_cap(int64_t n) { return (n + 3) / 4 * 4; }

int64_t kv_pages_ws_ints(int64_t num_pages, int64_t n) {
  const int64_t c = list_cap(num_pages), f = list_cap(n);
  return WS_LIST + std::max(3 * c, 6 * f);
}

template <int EDIT>
static cudaError_t launch_move(const KvLayers &l, const KvGeometry &g, const KvTableView &t,
                               int64_t max_copies, int64_t rows, int64_t cap, const int32_t *ws,
                               int32_t *d_status, cudaStream_t s) {
  const int64_t per = 2 * g.n_layers * (ceil_div<int64_t>(g.kv_bytes, MOVE_PIECE) +
                                        ceil_div<int64_t>(g.sc_bytes, MOVE_PIECE));
  const int64_t edits = rows * ceil_div<int64_t>(t.max_pages, EDIT_CHUNK);
  const int64_t blocks = std::min<int64_t>(std::max<int64_t>(std::max(max_copies * per, edits), 1),
                                           (int64_t)sm_count() * 8);
  return launch_pdl(k_kv_move<EDIT>, dim3((unsigned)blocks), dim3(MOVE_THREADS), 0, s, l, g, t, ws,
                    cap, d_status);
}

cudaError_t launch_kv_reserve(const KvTableView &t, int32_t num_pages, int32_t ps,
                              const int32_t *slots, const int32_t *n_new, int32_t n,
                              int32_t *d_status, cudaStream_t s) {
  static SmemOptIn opt_in;
  const size_t smem = plan_smem(num_pages, n);
  if (cudaError_t e = opt_in(k_kv_reserve, (int)smem)) return e;
  return launch_pdl(k_kv_reserve, dim3(1), dim3(PLAN_THREADS), smem, s, t, num_pages, ps, slots,
                    n_new, n, d_status);
}

cudaError_t launch_kv_free(const KvTableView &t, int32_t num_pages, int32_t ps,
                           const int32_t *slots, int64_t n, int32_t *d_status, cudaStream_t s) {
  return launch_pdl(k_kv_free, dim3((unsigned)n), dim3(256), 0, s, t, num_pages, ps, slots, d_status);
}

cudaError_t launch_kv_fork(const KvLayers &l, const KvGeometry &g, const KvTableView &t,
                           const int32_t *src, const int32_t *dst, int32_t n, int32_t *ws,
                           int32_t *d_status, cudaStream_t s) {
  static SmemOptIn opt_in;
  const size_t smem = plan_smem(g.src_pages, n);
  const int64_t cap = list_cap(n);
  if (cudaError_t e = opt_in(k_kv_fork_plan, (int)smem)) return e;
  if (cudaError_t e = launch_pdl(k_kv_fork_plan, dim3(1), dim3(PLAN_THREADS), smem, s, t,
                                 g.src_pages, g.page_size, src, dst, n, ws, cap, d_status))
    return e;
  return launch_move<EDIT_FORK>(l, g, t, n, n, cap, ws, d_status, s);
}

cudaError_t launch_kv_compact(const KvLayers &l, const KvGeometry &g, const KvTableView &t,
                              int32_t *n_used, int32_t *ws, int32_t *d_status, cudaStream_t s) {
  static SmemOptIn opt_in;
  const size_t smem = plan_smem(g.src_pages, 0);
  const int64_t cap = list_cap(g.src_pages);
  if (cudaError_t e = opt_in(k_kv_compact_plan, (int)smem)) return e;
  if (cudaError_t e = launch_pdl(k_kv_compact_plan, dim3(1), dim3(PLAN_THREADS), smem, s, t,
                                 g.src_pages, n_used, ws, cap))
    return e;
  return launch_move<EDIT_COMPACT>(l, g, t, g.src_pages / 2, t.n_slots, cap, ws, d_status, s);
}

cudaError_t launch_kv_copy(const KvLayers &l, const KvGeometry &g, bool same, const int32_t *src,
                           const int32_t *dst, int64_t n, int32_t *ws, int32_t *d_status,
                           cudaStream_t s) {
  static SmemOptIn opt_in;
  const size_t smem = (size_t)((g.dst_pages + 31) / 32) * 8;
  const int64_t cap = list_cap(n);
  const KvTableView none = {};
  if (cudaError_t e = opt_in(k_kv_copy_plan, (int)smem)) return e;
  if (cudaError_t e = launch_pdl(k_kv_copy_plan, dim3(1), dim3(PLAN_THREADS), smem, s, g.src_pages,
                                 g.dst_pages, same, src, dst, n, ws, cap, d_status))
    return e;
  return launch_move<EDIT_NONE>(l, g, none, n, 0, cap, ws, d_status, s);
}

}  // namespace bwta
