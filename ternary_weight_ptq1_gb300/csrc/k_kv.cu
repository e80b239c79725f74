// k_kv.cu -- key-value rows into a paged cache (quantised or rounded as they
// are written) and back out of it.
//
// A row is the head_dim values of one token and head.  PTQ_KV_I8 stores
//     s = max_d |x_d| / 127,  c_d = round_half_even(x_d / s)
// with IEEE fp32 divisions, so a row's codes and scale are a function of its
// values alone; the row stands for c_d s.  Both kernels move each byte once: HBM
// bounds them over bf16, the launch at a decode step's sizes.  Over int8 the write is
// bound by its instructions (420 of a warp, the SMs issue in 74% of their cycles;
// rintf and the conversions are a quarter of the slow pipe's time), the read waits for
// its loads.  A thread holds eight consecutive values (16 or 32
// bytes in, 8 or 16 out) of a key and the same of its value, so head_dim / 8
// neighbouring threads share a row and its maximum is three to five shuffles.
// (With two pieces of each the write and read of 33,001 x 4 x 256 took 139 us
// when this took 109.)
//
// Measured, a write and a read together, in CUDA graphs: 33,001 x 4 x 256, bf16, 82 us
// (98% of the copy rate); 8192 x 8 x 128, bf16 through int8, 25 us (61%); 64 x 8 x 128,
// fp32 through int8, 4.0 us, the launches.
#include "kv_row.cuh"

namespace ptq {
namespace {

constexpr int kThreads = 128;
using Geometry = CacheGeometry;

// Row r of T heads rows: head fastest, then token.
struct RowId {
  int64_t t;
  int h;
};
__device__ __forceinline__ RowId row_id(int64_t r, const Geometry& g) {
  if (r <= 0x7fffffff) {
    const int t = g.heads((int)r);
    return {t, (int)r - t * g.heads.d};
  }
  const int64_t t = r / g.heads.d;
  return {t, (int)(r - t * g.heads.d)};
}

template <Act T>
__device__ __forceinline__ void load8(const void* p, int64_t e, float (&x)[kVec]) {
  if constexpr (T == Act::F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <Act T>
__device__ __forceinline__ void store8(void* p, int64_t e, const float (&x)[kVec]) {
  if constexpr (T == Act::F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) =
        make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
  }
}

template <Act T, int D, bool kI8>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const void* __restrict__ k, const void* __restrict__ v, int64_t k_stride,
                    int64_t v_stride, const int32_t* __restrict__ slots, int64_t rows, Geometry g,
                    void* __restrict__ ck, void* __restrict__ cv, float* __restrict__ ks,
                    float* __restrict__ vs) {
  constexpr int kLanes = D / kVec;
  pdl_release();
  pdl_wait();
  const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int e = (int)(threadIdx.x % kLanes) * kVec;
  const bool in = r < rows;
  const RowId id = row_id(in ? r : 0, g);
  const int slot = in ? __ldg(slots + id.t) : -1;
  const bool ok = (unsigned)slot < (unsigned)g.pages_slots;
  float x[2][kVec] = {};
  if (ok) {
    load8<T>(k, id.t * k_stride + (int64_t)id.h * D + e, x[0]);
    load8<T>(v, id.t * v_stride + (int64_t)id.h * D + e, x[1]);
  }
  const int64_t row = ok ? cache_row(slot, id.h, g) : 0;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    void* to = n ? cv : ck;
    if constexpr (!kI8) {
      if (ok) store8<Act::BF16>(to, row * D + e, x[n]);
    } else {
      uint32_t w[2];
      const float s = quantise<kLanes, T == Act::F32, false>(x[n], w);  // (bf16 rows stay within 127 as they are)
      if (ok) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to) + row * D + e) = make_uint2(w[0], w[1]);
        if (e == 0) (n ? vs : ks)[row] = s;
      }
    }
  }
}

template <Act T, int D, bool kI8>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const void* __restrict__ ck, const void* __restrict__ cv,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   const int32_t* __restrict__ slots, int64_t rows, Geometry g,
                   void* __restrict__ k, void* __restrict__ v, int64_t k_stride, int64_t v_stride) {
  constexpr int kLanes = D / kVec;
  pdl_release();
  pdl_wait();
  const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int e = (int)(threadIdx.x % kLanes) * kVec;
  if (r >= rows) return;
  const RowId id = row_id(r, g);
  const int slot = __ldg(slots + id.t);
  float x[2][kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[0][i] = x[1][i] = __int_as_float(0x7fc00000);
  if ((unsigned)slot < (unsigned)g.pages_slots) {
    const int64_t row = cache_row(slot, id.h, g);
    if constexpr (!kI8) {
      load8<Act::BF16>(ck, row * D + e, x[0]);
      load8<Act::BF16>(cv, row * D + e, x[1]);
    } else {
      const uint2 wk = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(ck) + row * D + e);
      const uint2 wv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cv) + row * D + e);
      const float sk = ks[row], sv = vs[row];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        x[0][i] = (float)(int8_t)((i < 4 ? wk.x : wk.y) >> (8 * (i & 3))) * sk;
        x[1][i] = (float)(int8_t)((i < 4 ? wv.x : wv.y) >> (8 * (i & 3))) * sv;
      }
    }
  }
  store8<T>(k, id.t * k_stride + (int64_t)id.h * D + e, x[0]);
  store8<T>(v, id.t * v_stride + (int64_t)id.h * D + e, x[1]);
}

template <Act T, int D, bool kI8>
cudaError_t launch(const ptq_kv_cache& c, const KvRows& r, bool write, cudaStream_t st) {
  const Geometry g{(int)(c.pages * c.page_tokens), Divider(c.page_tokens), Divider(c.kv_heads)};
  const int64_t rows = r.T * c.kv_heads;
  const int64_t per = kThreads / (D / kVec), ctas = (rows + per - 1) / per;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas), block(kThreads);
  if (write)
    return launch_pdl(kv_write_kernel<T, D, kI8>, grid, block, 0, st, (const void*)r.k, (const void*)r.v,
                      r.k_stride, r.v_stride, r.slots, rows, g, c.k, c.v, c.k_scale, c.v_scale);
  return launch_pdl(kv_read_kernel<T, D, kI8>, grid, block, 0, st, (const void*)c.k, (const void*)c.v,
                    (const float*)c.k_scale, (const float*)c.v_scale, r.slots, rows, g, r.k, r.v,
                    r.k_stride, r.v_stride);
}

template <Act T, bool kI8>
cudaError_t by_dim(const ptq_kv_cache& c, const KvRows& r, bool write, cudaStream_t st) {
  switch (c.head_dim) {
    case 64: return launch<T, 64, kI8>(c, r, write, st);
    case 128: return launch<T, 128, kI8>(c, r, write, st);
    default: return launch<T, 256, kI8>(c, r, write, st);
  }
}

cudaError_t dispatch(const ptq_kv_cache& c, const KvRows& r, bool write, cudaStream_t st) {
  const bool i8 = c.type == PTQ_KV_I8;
  if (r.t == Act::F32) return i8 ? by_dim<Act::F32, true>(c, r, write, st) : by_dim<Act::F32, false>(c, r, write, st);
  return i8 ? by_dim<Act::BF16, true>(c, r, write, st) : by_dim<Act::BF16, false>(c, r, write, st);
}

}  // namespace

cudaError_t launch_kv_write(const ptq_kv_cache& c, const KvRows& r, cudaStream_t st) {
  return dispatch(c, r, true, st);
}
cudaError_t launch_kv_read(const ptq_kv_cache& c, const KvRows& r, cudaStream_t st) {
  return dispatch(c, r, false, st);
}

}  // namespace ptq
