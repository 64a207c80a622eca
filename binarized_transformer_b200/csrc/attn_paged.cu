// attn_paged.cu -- attention over the paged key-value cache.
//
// One warp a query row and head, one key after another: the running maximum m
// and sum l of the softmax and the weighted sum of the values are kept in fp32
// and rescaled by exp(m_old - m_new) when the maximum grows, so the keys are
// read once. The keys at positions [sink tiles) and [window ..) are walked in
// order; hidden ones are never read.
#include <algorithm>

#include "kv.cuh"

namespace bwta {

template <bool E4M3>
__device__ __forceinline__ float kv_value(const uint8_t *base, int64_t at) {
  if (E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)base[at]));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
  }
  return __half2float(reinterpret_cast<const __half *>(base)[at]);
}

template <bool E4M3>
__global__ void __launch_bounds__(128) k_attn_simple(const AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int64_t unit = ((int64_t)blockIdx.x * 128 + threadIdx.x) / 32;
  const int64_t row = unit / a.n_heads;
  const int h = (int)(unit - row * a.n_heads), kh = h / (a.n_heads / a.c.H);
  if (row >= (a.cu_q ? min((int64_t)a.cu_q[a.n_seq], a.total_q) : a.total_q)) return;
  const int64_t s = a.cu_q ? kv_find_seq(a.cu_q, a.n_seq, row) : row;
  bool bad = false;
  const int32_t slot = kv_slot(a.r, s);
  const int64_t len = kv_length(a.r, slot, a.c.ps, bad);
  const int64_t p = a.cu_q ? len - (a.cu_q[s + 1] - row) : len - 1;
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < a.c.D ? __half2float(__ushort_as_half(a.q[row * a.ldq + (int64_t)h * a.c.D + d])) : 0.0f;
  }
  const int64_t first = a.window ? max((int64_t)0, p - a.window + 1) : 0;
  for (int64_t j = 0; j <= p; ++j) {
    if (j < first && j >= a.sinks) j = first;
    const int32_t page = a.r.pages[(int64_t)slot * a.r.ld + j / a.c.ps];
    if ((uint32_t)page >= (uint32_t)a.c.num_pages) {
      bad = true;
      continue;
    }
    const int64_t kr = (int64_t)kh * a.c.ps + j % a.c.ps, at = (int64_t)page * a.c.page_stride + kr * a.c.D;
    const int64_t sat = (int64_t)page * a.c.scale_stride + kr;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.c.D) x = fmaf(q[i], kv_value<E4M3>(a.c.k, at + lane + 32 * i), x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(FULL, x, d);
    if (E4M3) x *= a.c.ks[sat];
    x *= a.scale;
    const float mn = fmaxf(m, x);
    const float c = m == mn ? 1.0f : expf(m - mn);
    float w = expf(x - mn);
    l = l * c + w;
    if (E4M3) w *= a.c.vs[sat];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.c.D) o[i] = fmaf(w, kv_value<E4M3>(a.c.v, at + lane + 32 * i), o[i] * c);
    m = mn;
  }
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane + 32 * i;
    if (d >= a.c.D) continue;
    const float y = p < 0 ? 0.0f : o[i] / l;
    finite &= y - y == 0.0f;
    a.out[row * a.ldo + (int64_t)h * a.c.D + d] = __half_as_ushort(__float2half_rn(y));
  }
  if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
  if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
}

cudaError_t launch_attn_simple(const AttnArgs &a, bool e4m3, cudaStream_t s) {
  const int64_t blocks = ceil_div<int64_t>(a.total_q * a.n_heads, 4);
  return launch_pdl(e4m3 ? k_attn_simple<true> : k_attn_simple<false>, dim3((unsigned)blocks),
                    dim3(128), 0, s, a);
}

}  // namespace bwta
