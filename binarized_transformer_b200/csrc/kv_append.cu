// kv_append.cu -- new tokens' keys and values into the pages of the cache.
//
// A row is one token's vector of one head. E4M3: the row's scale is 2^e with the
// smallest e for which max|x| <= 448 * 2^e; x * 2^-e is exact, so a value is
// rounded once, by the conversion. A group of 8, 16 or 32 lanes (4 elements
// each) holds one row of k and the same row of v, both loaded before either is
// used; the maximum is taken over the group in registers. One pass: bound by
// HBM (8 or 4 bytes read and 1 or 2 written an element), at the sizes of one
// decode step by the latency of kv_len -> page -> store. Measured (B200): 7 prompts,
// 10,600 tokens of 32 heads of 128, fp32 into fp16, 523 MB in 88 us (5.95 TB/s, 0.91 of
// a copy; with one head a group 128 us), into E4M3 106 us (0.63), fp16 rows into fp16 113
// (0.47: fewer bytes a load, the same lookups); 64 tokens of 8 heads into E4M3 4.2 us.
#include <algorithm>

#include "kv.cuh"

namespace bwta {

constexpr int AP_THREADS = 256;

// Exponent of the scale of a row whose largest magnitude has the fp32 bits b.
__device__ __forceinline__ int e4m3_row_exponent(uint32_t b) {
  if (b == 0) return 0;
  // 448 = 1.75 * 2^8: e = E - 8, one more if the significand is above 1.75.
  // (fp32 subnormals have E <= -127 and end at the lower limit.)
  const int E = (int)(b >> 23) - 127;
  const int e = E - 8 + ((b & 0x7fffffu) > 0x600000u);
  return min(max(e, -15), 8);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <bool F32>
__device__ __forceinline__ float4 load_row4(const void *p, int64_t at) {
  if (F32) return __ldcs(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + at));
  const uint2 h = __ldcs(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + at));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Write 4 elements of a row of k or v; returns false for a value that fp16 cannot hold.
template <int LPR, bool E4M3>
__device__ __forceinline__ bool store_row4(float4 x, uint8_t *base, float *scales, int64_t at,
                                           int64_t scale_at, int sub, bool live) {
  const float top4 = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
  // a NaN does not survive fmaxf: looked for by itself (x - x is 0 for every finite x)
  const bool nan = !(x.x - x.x == 0.0f && x.y - x.y == 0.0f && x.z - x.z == 0.0f && x.w - x.w == 0.0f);
  if (E4M3) {
    uint32_t top = live ? __float_as_uint(top4) : 0u;
#pragma unroll
    for (int d = LPR / 2; d > 0; d /= 2) top = max(top, __shfl_xor_sync(FULL, top, d));
    const int e = e4m3_row_exponent(top);
    if (live) {
      const float up = __uint_as_float((uint32_t)(127 - e) << 23), lim = e == 8 ? 240.0f : 448.0f;
      auto f = [&](float v) { return fminf(fmaxf(v * up, -lim), lim); };
      *reinterpret_cast<uint32_t *>(base + at) = e4m3x4(f(x.x), f(x.y), f(x.z), f(x.w));
      if (sub == 0) scales[scale_at] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
  } else if (live) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(base + at * 2) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
  return !live || (!nan && top4 < 65520.0f);
}

// A group of LPR lanes takes HB heads of one token at a time: where they go is looked
// up once, and all their loads are under way before the first is used.
template <int LPR, int HB, bool F32, bool E4M3>
__global__ void __launch_bounds__(AP_THREADS) k_kv_append(const KvAppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int sub = threadIdx.x % LPR, d = sub * 4;
  const int64_t group = ((int64_t)blockIdx.x * AP_THREADS + threadIdx.x) / LPR;
  const int64_t groups = (int64_t)gridDim.x * AP_THREADS / LPR;
  const int hb = (a.c.H + HB - 1) / HB;
  const int64_t work = (a.cu_q ? (int64_t)min((int64_t)a.cu_q[a.n_seq], a.total_q) : a.total_q) * hb;
  bool bad = false, finite = true;
  const int64_t rounds = ceil_div<int64_t>(work, groups);
  for (int64_t i = 0; i < rounds; ++i) {  // every lane of a warp takes every round: shuffles inside
    const int64_t r = i * groups + group;
    const bool in = r < work;
    const int64_t tok = in ? r / hb : 0;
    const int h0 = in ? (int)(r - tok * hb) * HB : 0;
    float4 xk[HB], xv[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      xk[j] = xv[j] = make_float4(0, 0, 0, 0);
      if (in && h0 + j < a.c.H && d < a.c.D) {
        xk[j] = load_row4<F32>(a.k, tok * a.ldk + (int64_t)(h0 + j) * a.c.D + d);
        xv[j] = load_row4<F32>(a.v, tok * a.ldv + (int64_t)(h0 + j) * a.c.D + d);
      }
    }
    bool live = in && d < a.c.D;
    int64_t at = 0, sat = 0;
    if (in) {
      const int64_t s = a.cu_q ? kv_find_seq(a.cu_q, a.n_seq, tok) : tok;
      const int32_t slot = kv_slot(a.r, s);
      int64_t pos = -1;
      if (slot >= 0) pos = a.cu_q ? (int64_t)a.r.len[slot] - (a.cu_q[s + 1] - tok) : (int64_t)a.r.len[slot] - 1;
      const int64_t idx = pos < 0 ? a.r.max_pages : pos / a.c.ps;
      int32_t page = -1;
      if (idx < a.r.max_pages) page = a.r.pages[(int64_t)slot * a.r.ld + idx];
      if ((uint32_t)page >= (uint32_t)a.c.num_pages) {
        bad = true;
        live = false;
      } else {
        const int64_t row = (int64_t)h0 * a.c.ps + (pos - idx * a.c.ps);
        at = (int64_t)page * a.c.page_stride + row * a.c.D + d;
        sat = (int64_t)page * a.c.scale_stride + row;
      }
    }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      const bool on = live && h0 + j < a.c.H;
      const int64_t to = at + (int64_t)j * a.c.ps * a.c.D, sto = sat + (int64_t)j * a.c.ps;
      finite &= store_row4<LPR, E4M3>(xk[j], const_cast<uint8_t *>(a.c.k), const_cast<float *>(a.c.ks), to, sto, sub, on);
      finite &= store_row4<LPR, E4M3>(xv[j], const_cast<uint8_t *>(a.c.v), const_cast<float *>(a.c.vs), to, sto, sub, on);
    }
  }
  if (bad) flag_status(a.d_status, BWTA_STATUS_BAD_PAGE);
  if (!finite) flag_status(a.d_status, BWTA_STATUS_NONFINITE);
}

template <int LPR, int HB>
static cudaError_t launch_append_t(const KvAppendArgs &a, int sms, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>(
      ceil_div<int64_t>(a.total_q * ceil_div(a.c.H, HB) * LPR, AP_THREADS), (int64_t)sms * 8);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(AP_THREADS), 0, s, a);
  };
  if (a.f32) return a.e4m3 ? go(k_kv_append<LPR, HB, true, true>) : go(k_kv_append<LPR, HB, true, false>);
  return a.e4m3 ? go(k_kv_append<LPR, HB, false, true>) : go(k_kv_append<LPR, HB, false, false>);
}

template <int LPR>
static cudaError_t launch_append_rows(const KvAppendArgs &a, cudaStream_t s) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  sms = std::max(sms, 1);
  // Several heads a group once every SM has its warps: below, one head each is the shorter way.
  const bool many = a.total_q * a.c.H * LPR >= (int64_t)sms * 2048 * 4;
  return many ? launch_append_t<LPR, 4>(a, sms, s) : launch_append_t<LPR, 1>(a, sms, s);
}

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s) {
  if (a.c.D <= 32) return launch_append_rows<8>(a, s);
  if (a.c.D <= 64) return launch_append_rows<16>(a, s);
  return launch_append_rows<32>(a, s);
}

}  // namespace bwta
