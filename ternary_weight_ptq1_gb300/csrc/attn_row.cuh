// attn_row.cuh -- attention of one query row, a warp at a time: lane l holds
// the values [l D/32, (l + 1) D/32) of the query, a key, a value and the
// output, a score is a shuffle sum, and the softmax is kept as a running
// maximum m and sum l (base 2):
//     m' = max(m, s),  a = 2^(m - m'),  p = 2^(s - m'),
//     l = l a + p,  o = o a + p v.
// fp32 throughout.
#pragma once

#include <stdint.h>

namespace ptq {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct RowState {
  float m = kNegInf, l = 0.0f;
  float o[D / 32] = {};

  // One more key and value; scale2 = softmax scale * log2(e).
  __device__ __forceinline__ void add(const float (&q)[D / 32], const float (&k)[D / 32],
                                      const float (&v)[D / 32], float scale2) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
    s *= scale2;
    const float mn = fmaxf(m, s);  // a NaN score leaves m and makes p NaN
    const float a = mn == kNegInf ? 1.0f : exp2f(m - mn);
    const float p = s == kNegInf ? 0.0f : exp2f(s - mn);
    m = mn;
    l = fmaf(l, a, p);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], a, p * v[i]);
  }

  // The state of both of two disjoint sets of keys.
  __device__ __forceinline__ void join(float m2, float l2, const float (&o2)[D / 32]) {
    // l = 0: no key so far, o = 0.  A NaN score leaves m alone and makes l
    // and o NaN, which stay.
    const float mn = fmaxf(m, m2);
    const float a = l == 0.0f ? 0.0f : m == kNegInf ? 1.0f : exp2f(m - mn);
    const float b = l2 == 0.0f ? 0.0f : m2 == kNegInf ? 1.0f : exp2f(m2 - mn);
    m = mn;
    l = l * a + l2 * b;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * a + o2[i] * b;
  }
};

}  // namespace ptq
