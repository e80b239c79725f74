// k_attn_chunk.cu -- attention of chunks of new tokens over their paged
// key-value cache, all of it or a sliding window and the first tokens.
//
//   s_j = scale q . k_j,  p_j = 2^(s_j log2(e) - m),  out = sum_j p_j v_j / sum_j p_j
//
// over the tokens j <= p of the query's position p, with a window those with
// p - window < j or j < sinks.  A warp a query row: 32 keys at a time, a lane's
// own key for the scores and its own columns for the output.
#include <cuda_bf16.h>

#include "attn_row.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ int clamped(int v, int hi) { return min(max(v, 0), hi); }

// Eight consecutive values of a cached row, in fp32 (int8: times its scale).
template <bool kI8>
__device__ __forceinline__ void row8(const void* p, int64_t e, float scale, float (&x)[8]) {
  if constexpr (kI8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + e));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3))) * scale;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <int D, bool kI8>
__global__ void __launch_bounds__(32 * kWarps) attn_chunk_kernel(ChunkArgs a) {
  constexpr int N = D / 32;
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= a.Tq * a.Hq) return;
  const int t = (int)(r / a.Hq), hq = (int)(r - (int64_t)t * a.Hq);
  const int Tq = (int)a.Tq, ps = (int)a.c.page_tokens, heads = (int)a.c.kv_heads;
  const int h = hq / (int)(a.Hq / heads);
  int lo = 0, hi = (int)a.B;  // the last sequence that begins at t or before
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (clamped(__ldg(a.cu_q + mid), Tq) <= t) lo = mid; else hi = mid;
  }
  const int q0 = clamped(__ldg(a.cu_q + lo), Tq), q1 = clamped(__ldg(a.cu_q + lo + 1), Tq);
  if (t < q0 || t >= q1) return;
  const int64_t most = a.table_width * ps;
  const int n = __ldg(a.lens + lo);
  const int len = n < 0 ? 0 : n > most ? (int)most : n;
  const int p = len - q1 + t, end = max(0, p + 1);
  const int from = a.window ? max(0, end - a.window) : 0;
  const int skip = max(0, from - a.sinks), seen = end - skip;
  RowState<D> s;
  float l, small = 1.0f;
  // The weights' sum may be large, and the sums of values near the largest overflow
  // although their mean does not: then again with smaller weights.
  for (int again = 0; again < 2; ++again) {
    s = RowState<D>();
    for (int j0 = 0; j0 < seen; j0 += 32) {
      int64_t row = -1;
      bool bad = false;
      int j = j0 + lane;
      if (j < seen) {
        j += j >= a.sinks ? skip : 0;
        const int page = __ldg(a.table + (int64_t)lo * a.table_width + j / ps);
        bad = (unsigned)page >= (unsigned)a.c.pages;
        if (!bad) row = ((int64_t)page * heads + h) * ps + j % ps;
      }
      float x = kNegInf, vs = 0.0f;
      if (row >= 0) {
        x = 0.0f;
        for (int d = 0; d < D; d += 8) {
          float kx[8], qx[8];
          row8<kI8>(a.c.k, row * D + d, 1.0f, kx);
          row8<false>(a.q, t * a.q_stride + (int64_t)hq * D + d, 1.0f, qx);
#pragma unroll
          for (int i = 0; i < 8; ++i) x = fmaf(kx[i], qx[i], x);
        }
        if constexpr (kI8) {
          x *= __ldg(a.c.k_scale + row);
          vs = __ldg(a.c.v_scale + row);
        }
        x *= a.scale * kLog2e;
      }
      if (bad) x = __int_as_float(0x7fc00000);
      const float w = s.weigh(x);
      for (int i = 0; i < min(32, seen - j0); ++i) {
        const float wi = __shfl_sync(~0u, w, i), si = __shfl_sync(~0u, vs, i);
        const int64_t ri = __shfl_sync(~0u, row, i);
        if (ri < 0) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float v;
          if constexpr (kI8)
            v = (float)static_cast<const int8_t*>(a.c.v)[ri * D + lane * N + e] * si;
          else
            v = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.c.v)[ri * D + lane * N + e] << 16);
          s.o[e] = fmaf(wi * small, v, s.o[e]);
        }
      }
    }
    l = s.l;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(~0u, l, i);
    bool fine = true;
#pragma unroll
    for (int e = 0; e < N; ++e) fine = fine && fabsf(s.o[e]) < -kNegInf;
    if (!(l == l) || __all_sync(~0u, fine) || again) break;
    small = 0x1p-40f;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / small / l;
#pragma unroll
  for (int e = 0; e < N; ++e)
    a.out[r * D + lane * N + e] = __bfloat16_as_ushort(__float2bfloat16_rn(l == l ? s.o[e] * inv : l));
  if (a.lse && lane == 0) a.lse[r] = l == 0.0f ? kNegInf : s.m * kLn2 + logf(l);
}

template <bool kI8>
cudaError_t by_dim(const ChunkArgs& a, cudaStream_t st) {
  const int64_t ctas = (a.Tq * a.Hq + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas), block(32 * kWarps);
  switch (a.c.head_dim) {
    case 64: return launch_pdl(attn_chunk_kernel<64, kI8>, grid, block, 0, st, a);
    case 128: return launch_pdl(attn_chunk_kernel<128, kI8>, grid, block, 0, st, a);
    default: return launch_pdl(attn_chunk_kernel<256, kI8>, grid, block, 0, st, a);
  }
}

}  // namespace

size_t attn_chunk_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attn_chunk(const ChunkArgs& a, void*, cudaStream_t st) {
  return a.c.type == PTQ_KV_I8 ? by_dim<true>(a, st) : by_dim<false>(a, st);
}

}  // namespace ptq
