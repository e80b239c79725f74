// k_attn_prefill.cu -- attention of packed prompts.  One warp per (query,
// head), over the keys it sees.
#include <cuda_bf16.h>

#include "attn_row.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kWarps = 4;

template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float((uint32_t)__ldg(p + i) << 16);
}

__device__ __forceinline__ int clamped(int v, int64_t hi) {
  return v < 0 ? 0 : v > hi ? (int)hi : v;
}

// One query row: query t of the packed queries, head hq, of sequence b.
template <int D>
__device__ void attend_row(const PrefillArgs& a, int b, int t, int hq, int lane) {
  constexpr int N = D / 32;
  const int q0 = clamped(a.cu_q[b], a.Tq), q1 = clamped(a.cu_q[b + 1], a.Tq);
  const int k0 = clamped(a.cu_k[b], a.Tk), k1 = clamped(a.cu_k[b + 1], a.Tk);
  const int h = hq / (int)(a.Hq / a.Hkv);
  int end = k1;
  if (a.causal) end = min(k1, k1 - (q1 - q0) + (t - q0) + 1);
  float q[N];
  load_bf16(a.q + (int64_t)t * a.q_stride + (int64_t)hq * D + lane * N, q);
  RowState<D> r;
  for (int j = k0; j < end; ++j) {
    float k[N], v[N];
    load_bf16(a.k + (int64_t)j * a.k_stride + (int64_t)h * D + lane * N, k);
    load_bf16(a.v + (int64_t)j * a.v_stride + (int64_t)h * D + lane * N, v);
    r.add(q, k, v, a.scale * kLog2e);
  }
  const int64_t row = (int64_t)t * a.Hq + hq;
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;
  if (a.lse && lane == 0) a.lse[row] = r.l == 0.0f ? kNegInf : r.m * kLn2 + logf(r.l);
#pragma unroll
  for (int i = 0; i < N; ++i)
    a.out[row * D + lane * N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(r.o[i] * inv));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_prefill_kernel(PrefillArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + warp;
  if (i >= a.Tq * a.Hq) return;
  const int t = (int)(i / a.Hq), hq = (int)(i % a.Hq);
  for (int b = 0; b < a.B; ++b)  // the sequence that holds query t, if one does
    if (t >= clamped(a.cu_q[b], a.Tq) && t < clamped(a.cu_q[b + 1], a.Tq)) {
      attend_row<D>(a, b, t, hq, lane);
      return;
    }
}

template <int D>
cudaError_t launch(const PrefillArgs& a, cudaStream_t st) {
  const int64_t ctas = (a.Tq * a.Hq + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  attn_prefill_kernel<D><<<(unsigned)ctas, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t attn_prefill_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attn_prefill(const PrefillArgs& a, void*, cudaStream_t st) {
  switch (a.D) {
    case 64: return launch<64>(a, st);
    case 128: return launch<128>(a, st);
    default: return launch<256>(a, st);
  }
}

}  // namespace ptq
