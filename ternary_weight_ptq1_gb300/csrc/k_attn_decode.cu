// k_attn_decode.cu -- attention of one new token of each sequence over its
// paged key-value cache.  One CTA per (sequence, query head); its warps take
// the tokens in turn and their states are joined at the end.
#include <cuda_bf16.h>

#include "attn_row.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kWarps = 8;

template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float((uint32_t)__ldg(p + i) << 16);
}

template <Act T, int D, bool kI8>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(DecodeArgs a) {
  constexpr int N = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, hq = blockIdx.x, h = hq / (int)(a.Hq / a.c.kv_heads);
  const int ps = (int)a.c.page_tokens;
  const int64_t most = a.table_width * a.c.page_tokens;
  int len = a.lens[b];
  len = len < 0 ? 0 : len > most ? (int)most : len;
  float q[N];
  const int64_t at = (int64_t)b * a.q_stride + (int64_t)hq * D + lane * N;
  if constexpr (T == Act::F32) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = static_cast<const float*>(a.q)[at + i];
  } else {
    load_bf16(static_cast<const uint16_t*>(a.q) + at, q);
  }
  RowState<D> r;
  for (int j = warp; j < len; j += kWarps) {
    const int page = a.table[(int64_t)b * a.table_width + j / ps];
    float k[N], v[N];
    if ((unsigned)page >= (unsigned)a.c.pages) {
#pragma unroll
      for (int i = 0; i < N; ++i) k[i] = v[i] = __int_as_float(0x7fc00000);
    } else {
      const int64_t row = ((int64_t)page * a.c.kv_heads + h) * ps + j % ps;
      if constexpr (kI8) {
        const float ks = a.c.k_scale[row], vs = a.c.v_scale[row];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          k[i] = (float)static_cast<const int8_t*>(a.c.k)[row * D + lane * N + i] * ks;
          v[i] = (float)static_cast<const int8_t*>(a.c.v)[row * D + lane * N + i] * vs;
        }
      } else {
        load_bf16(static_cast<const uint16_t*>(a.c.k) + row * D + lane * N, k);
        load_bf16(static_cast<const uint16_t*>(a.c.v) + row * D + lane * N, v);
      }
    }
    r.add(q, k, v, a.scale * kLog2e);
  }
  if (lane == 0) {
    sm[warp] = r.m;
    sl[warp] = r.l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) so[warp][lane * N + i] = r.o[i];
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < kWarps; ++w) {
    float o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = so[w][lane * N + i];
    r.join(sm[w], sl[w], o);
  }
  const int64_t row = (int64_t)b * a.Hq + hq;
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;
  if (a.lse && lane == 0) a.lse[row] = r.l == 0.0f ? kNegInf : r.m * kLn2 + logf(r.l);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = r.o[i] * inv;
    if constexpr (T == Act::F32)
      static_cast<float*>(a.out)[row * D + lane * N + i] = y;
    else
      static_cast<__nv_bfloat16*>(a.out)[row * D + lane * N + i] = __float2bfloat16_rn(y);
  }
}

template <Act T, int D, bool kI8>
cudaError_t launch(const DecodeArgs& a, cudaStream_t st) {
  if (a.B > 65535) return cudaErrorInvalidValue;
  attn_decode_kernel<T, D, kI8><<<dim3((unsigned)a.Hq, (unsigned)a.B), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template <Act T, bool kI8>
cudaError_t by_dim(const DecodeArgs& a, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch<T, 64, kI8>(a, st);
    case 128: return launch<T, 128, kI8>(a, st);
    default: return launch<T, 256, kI8>(a, st);
  }
}

}  // namespace

size_t attn_decode_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attn_decode(const DecodeArgs& a, void*, cudaStream_t st) {
  const bool i8 = a.c.type == PTQ_KV_I8;
  if (a.t == Act::F32) return i8 ? by_dim<Act::F32, true>(a, st) : by_dim<Act::F32, false>(a, st);
  return i8 ? by_dim<Act::BF16, true>(a, st) : by_dim<Act::BF16, false>(a, st);
}

}  // namespace ptq
