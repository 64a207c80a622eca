// kv.cuh -- views of the paged key-value cache and its table for the kernels,
// and the launchers of the calls on them (validated in kv_abi.cu).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace bwta {

constexpr int KV_MAX_D = 128;

// The softmax's weights are 2^(x - m), rounded to fp16 for the product with V. The
// reference m is set ATTN_HEAD below the maximum seen so far and follows it when a
// score passes m by more than ATTN_SLACK (log2), so the weights use all of fp16's
// range: up to 2^15, and down to 2^-21 of the largest before they lose bits and 2^-32
// before they vanish. (With m at the maximum the small weights of a long row behind
// one dominant key are lost while their sum counts them: of 32,768 keys behind a first
// one with 99.9% of the weight and no value, a fifth of the output.)
constexpr float ATTN_HEAD = 7.0f, ATTN_SLACK = 15.0f;

// A mean of fp16 values on its way to fp16. Rounded weights over the sum of unrounded
// ones can pass the largest value by 2^-11 of it, and fp16 has nothing above 65504 but
// Inf. Inf and NaN stay as they are.
__device__ __forceinline__ float mean_to_f16_range(float x) {
  return fabsf(x) < 131072.0f ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x;
}

// One layer's pool. Strides in elements of k / v and in floats of the scales.
struct KvView {
  const uint8_t *k, *v;
  const float *ks, *vs;
  int64_t page_stride, scale_stride;
  int32_t num_pages, ps, H, D;
};

struct KvRows {
  const int32_t *pages;
  const int32_t *len;
  const int32_t *slots;  // NULL: sequence s is slot s
  int64_t ld;
  int32_t max_pages, n_slots;
};

// Slot of sequence s, or -1 when it is outside the table.
__device__ __forceinline__ int32_t kv_slot(const KvRows &r, int64_t s) {
  if (!r.slots) return (int32_t)s;
  const int32_t v = r.slots[s];
  return (uint32_t)v < (uint32_t)r.n_slots ? v : -1;
}

// Tokens of a slot, cut to its row of pages; sets bad when it had to cut.
__device__ __forceinline__ int32_t kv_length(const KvRows &r, int32_t slot, int32_t ps, bool &bad) {
  if (slot < 0) {
    bad = true;
    return 0;
  }
  const int32_t len = r.len[slot];
  const int64_t room = (int64_t)r.max_pages * ps;
  if (len < 0 || len > room) {
    bad = true;
    return len < 0 ? 0 : (int32_t)room;
  }
  return len;
}

// The sequence whose rows [cu[s], cu[s+1]) hold row t, for cu[0] <= t < cu[n].
__device__ __forceinline__ int64_t kv_find_seq(const int32_t *cu, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// a / b for a >= 0, b > 0; a division in 64 bits takes several times as long.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// ---- blocks of a cluster
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What lies at shared-memory address `at` of block `rank` of the cluster.
__device__ __forceinline__ float2 cluster_ld2(uint32_t at, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t at, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

struct AttnArgs {
  KvView c;
  KvRows r;
  const int32_t *cu_q;  // NULL: one row each
  int64_t n_seq, total_q;
  const uint16_t *q;
  int64_t ldq;
  int32_t n_heads;
  float scale;
  int64_t window, sinks;
  uint16_t *out;
  int64_t ldo;
  int32_t *d_status;
};

struct KvAppendArgs {
  KvView c;
  KvRows r;
  const int32_t *cu_q;
  int64_t n_seq, total_q;
  const void *k, *v;
  int64_t ldk, ldv;
  bool f32, e4m3;
  int32_t *d_status;
};

// One layer's buffers in a page call.
struct KvLayer {
  uint8_t *k, *v;
  float *ks, *vs;
};
struct KvLayers {
  KvLayer src[BWTA_KV_MAX_LAYERS];
  KvLayer dst[BWTA_KV_MAX_LAYERS];
};
struct KvGeometry {
  int64_t kv_bytes;         // of one page of k (or v)
  int64_t src_kv_stride, dst_kv_stride;  // bytes between pages
  int64_t sc_bytes, src_sc_stride, dst_sc_stride;  // the same for the scales; 0: none
  int32_t n_layers, src_pages, dst_pages, page_size;
};
struct KvTableView {
  int32_t *pages, *len, *ref;
  int64_t ld;
  int32_t max_pages, n_slots;
};

int64_t attn_decode_ws(int64_t n_heads, int64_t n_kv_heads, int64_t head_dim);
cudaError_t launch_attn_decode(const AttnArgs &a, bool e4m3, float *ws, cudaStream_t s);
int64_t kv_pages_ws_ints(int64_t num_pages, int64_t n);
cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s);
int64_t attn_prompt_blocks(int64_t n_seq, int64_t total_q, int64_t n_heads, int64_t n_kv_heads);
cudaError_t launch_attn_prompt(const AttnArgs &a, bool e4m3, cudaStream_t s);
cudaError_t launch_kv_reserve(const KvTableView &t, int32_t num_pages, int32_t ps,
                              const int32_t *slots, const int32_t *n_new, int32_t n,
                              int32_t *d_status, cudaStream_t s);
cudaError_t launch_kv_free(const KvTableView &t, int32_t num_pages, int32_t ps,
                           const int32_t *slots, int64_t n, int32_t *d_status, cudaStream_t s);
cudaError_t launch_kv_fork(const KvLayers &l, const KvGeometry &g, const KvTableView &t,
                           const int32_t *src, const int32_t *dst, int32_t n, int32_t *ws,
                           int32_t *d_status, cudaStream_t s);
cudaError_t launch_kv_compact(const KvLayers &l, const KvGeometry &g, const KvTableView &t,
                              int32_t *n_used, int32_t *ws, int32_t *d_status, cudaStream_t s);
cudaError_t launch_kv_copy(const KvLayers &l, const KvGeometry &g, bool same, const int32_t *src,
                           const int32_t *dst, int64_t n, int32_t *ws, int32_t *d_status,
                           cudaStream_t s);

}  // namespace bwta
