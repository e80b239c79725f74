// kv_row.cuh -- eight values of a key or value row in a thread, as the paged
// cache's kernels hold them: loads, stores, and the int8 codes of a row that
// neighbouring threads share.
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include "packed.cuh"
#include "ptq_internal.cuh"

namespace ptq {

constexpr int kVec = 8;  // values a thread holds of a row

// Where a row of the cache is, and which row of T heads rows a thread has.
struct CacheGeometry {
  int pages_slots;  // pages * page_tokens
  Divider page_tokens, heads;
};

// The row of the cache that (slot, h) names, in units of rows.
__device__ __forceinline__ int64_t cache_row(int slot, int h, const CacheGeometry& g) {
  const int page = g.page_tokens(slot), p = slot - page * g.page_tokens.d;
  return ((int64_t)page * g.heads.d + h) * g.page_tokens.d + p;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// round_half_even(x / s) for |x| <= 127 s, given r near 1 / s: x r is within
// 1e-4 of the quotient, and where that leaves the rounding open (or r is not
// finite) the division decides.
__device__ __forceinline__ int code_of(float x, float s, float r) {
  const float t = x * r;
  float n = rintf(t);
  if (!(fabsf(t - n) < 0.4999f)) n = rintf(x / s);
  return (int)n;
}

// The same of eight values at once: x r + 1.5 2^23 has its nearest integer in its low byte,
// and where one is not clear of a half the divisions decide for all.
__device__ __forceinline__ void codes_of(const float (&x)[kVec], float s, float r, uint32_t (&w)[2]) {
  const uint64_t rr = pair(r, r), magic = pair(12582912.0f, 12582912.0f), back = pair(-12582912.0f, -12582912.0f);
  uint32_t c[kVec], off = 0;  // off: from the nearest integer, its bits (NaN is the largest)
#pragma unroll
  for (int i = 0; i < kVec; i += 2) {
    const uint64_t y = fma2(pair(x[i], x[i + 1]), rr, magic);
    float n0, n1, d0, d1, y0, y1;
    unpair(add2(y, back), n0, n1);
    unpair(fma2(pair(x[i], x[i + 1]), rr, pair(-n0, -n1)), d0, d1);
    unpair(y, y0, y1);
    off = max(off, max(__float_as_uint(d0) & 0x7fffffffu, __float_as_uint(d1) & 0x7fffffffu));
    c[i] = __float_as_uint(y0), c[i + 1] = __float_as_uint(y1);
  }
  if (__builtin_expect(off >= __float_as_uint(0.4999f), 0)) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) c[i] = (uint32_t)(int)rintf(x[i] / s);
  }
#pragma unroll
  for (int i = 0; i < kVec; i += 4)
    w[i / 4] = __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
}

// The scale and the codes (w, a byte each) of a row whose kLanes neighbouring
// threads hold eight values each.  kTiny: the scale may be subnormal.  kEight: all codes
// at once, the same ones (kv_append of 20,011 x 4 x 256, with its queries, and the way back
// 156 us for 168; kv_write, which waits for other things, 25.8 for 25.3 at 8192 x 8 x 128).
template <int kLanes, bool kTiny, bool kEight>
__device__ __forceinline__ float quantise(float (&x)[kVec], uint32_t (&w)[2]) {
  float m = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    m = fmaxf(m, fabsf(x[i]));
    bad |= !(fabsf(x[i]) < __int_as_float(0x7f800000));
  }
  if (bad) m = __int_as_float(0x7f800000);  // fmaxf drops NaN: a non-finite row is infinite
#pragma unroll
  for (int i = kLanes / 2; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, i));
  const bool finite = m < __int_as_float(0x7f800000);
  const float s = finite ? m / 127.0f : __int_as_float(0x7fc00000);
  w[0] = w[1] = 0;
  if (s > 0.0f) {  // a row of zeros (or of values whose scale underflows) keeps zero codes
    // A scale of few bits is rounded by up to half of itself, and the row's
    // largest values may pass 127 s: their codes are 127.  (The smallest bf16
    // value, 2^16 units, gives a scale of 516: at most 127.2 of it.)
    if constexpr (kTiny) {
      if (__builtin_expect(s < FLT_MIN, 0)) {
        asm volatile("");  // a branch: as selections they take 3% of the write's time
        const float lim = 127.0f * s;
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = fminf(fmaxf(x[i], -lim), lim);
      }
    }
    const float inv = 1.0f / s;
    if constexpr (kEight) {
      codes_of(x, s, inv, w);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[i >> 2] |= ((uint32_t)code_of(x[i], s, inv) & 0xffu) << (8 * (i & 3));
    }
  }
  return s;
}

}  // namespace ptq
