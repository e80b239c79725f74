// attn_row.cuh -- attention of one query row by a warp: lane l holds the columns
// [l D/32, (l + 1) D/32) of the output, a key's score is one lane's, and the
// softmax is kept as a running maximum m and sum l (base 2):
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

  // 32 more keys, a score in units of log2 a lane: the lane's weight, which is in l
  // (the lane's share of the sum) but not yet in o.
  __device__ __forceinline__ float weigh(float s) {
    float mn = fmaxf(m, s);  // a NaN score leaves m and makes its weight NaN
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mn = fmaxf(mn, __shfl_xor_sync(~0u, mn, i));
    const float a = mn == kNegInf ? 1.0f : exp2f(m - mn);
    const float p = s == kNegInf ? 0.0f : exp2f(s - mn);
    m = mn;
    l = fmaf(l, a, p);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= a;
    return p;
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
