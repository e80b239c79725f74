// k_kv.cu -- key-value rows into a paged cache (quantised or rounded as they
// are written) and back out of it.
//
// A row is the head_dim values of one token and head.  PTQ_KV_I8 stores
//     s = max_d |x_d| / 127,  c_d = round_half_even(x_d / s)
// with IEEE fp32 divisions, so a row's codes and scale are a function of its
// values alone; the row stands for c_d s.  Both kernels move each byte once
// and compute a few operations a value: HBM bounds them, the launch at a
// decode step's sizes.  A thread holds eight consecutive values (16 or 32
// bytes in, 8 or 16 out), so head_dim / 8 neighbouring threads share a row
// and its maximum is three to five shuffles.
#include <cuda_bf16.h>

#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;  // values a thread holds of a row

struct Geometry {
  int pages_slots;  // pages * page_tokens
  int page_tokens, heads;
};

// Row r of 2 T heads rows: head fastest, then key (0) or value (1), then token.
struct RowId {
  int64_t t;
  int h, kv;
};
__device__ __forceinline__ RowId row_id(int64_t r, int heads) {
  const int64_t q = r / heads;
  return {q >> 1, (int)(r - q * heads), (int)(q & 1)};
}

// The row of the cache that (slot, h) names, in units of rows.
__device__ __forceinline__ int64_t cache_row(int slot, int h, const Geometry& g) {
  const int page = slot / g.page_tokens, p = slot - page * g.page_tokens;
  return ((int64_t)page * g.heads + h) * g.page_tokens + p;
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

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
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
  const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int e = (int)(threadIdx.x % kLanes) * kVec;
  const bool in = r < rows;
  const RowId id = row_id(in ? r : 0, g.heads);
  const int slot = in ? __ldg(slots + id.t) : -1;
  const bool ok = (unsigned)slot < (unsigned)g.pages_slots;
  float x[kVec] = {};
  if (ok) load8<T>(id.kv ? v : k, id.t * (id.kv ? v_stride : k_stride) + (int64_t)id.h * D + e, x);
  if constexpr (!kI8) {
    if (ok) store8<Act::BF16>(id.kv ? cv : ck, cache_row(slot, id.h, g) * D + e, x);
  } else {
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
    if (!ok) return;
    const bool finite = m < __int_as_float(0x7f800000);
    const float s = finite ? m / 127.0f : __int_as_float(0x7fc00000);
    uint32_t w[2] = {0, 0};
    if (s > 0.0f) {  // a row of zeros (or of values whose scale underflows) keeps zero codes
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        w[i >> 2] |= ((uint32_t)__float2int_rn(x[i] / s) & 0xffu) << (8 * (i & 3));
    }
    const int64_t row = cache_row(slot, id.h, g);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(id.kv ? cv : ck) + row * D + e) =
        make_uint2(w[0], w[1]);
    if (e == 0) (id.kv ? vs : ks)[row] = s;
  }
}

template <Act T, int D, bool kI8>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const void* __restrict__ ck, const void* __restrict__ cv,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   const int32_t* __restrict__ slots, int64_t rows, Geometry g,
                   void* __restrict__ k, void* __restrict__ v, int64_t k_stride, int64_t v_stride) {
  constexpr int kLanes = D / kVec;
  const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int e = (int)(threadIdx.x % kLanes) * kVec;
  if (r >= rows) return;
  const RowId id = row_id(r, g.heads);
  const int slot = __ldg(slots + id.t);
  float x[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[i] = __int_as_float(0x7fc00000);
  if ((unsigned)slot < (unsigned)g.pages_slots) {
    const int64_t row = cache_row(slot, id.h, g);
    if constexpr (!kI8) {
      load8<Act::BF16>(id.kv ? cv : ck, row * D + e, x);
    } else {
      const uint2 w =
          *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(id.kv ? cv : ck) + row * D + e);
      const float s = (id.kv ? vs : ks)[row];
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        x[i] = (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * s;
    }
  }
  store8<T>(id.kv ? v : k, id.t * (id.kv ? v_stride : k_stride) + (int64_t)id.h * D + e, x);
}

template <Act T, int D, bool kI8>
cudaError_t launch(const ptq_kv_cache& c, const KvRows& r, bool write, cudaStream_t st) {
  const Geometry g{(int)(c.pages * c.page_tokens), (int)c.page_tokens, (int)c.kv_heads};
  const int64_t rows = 2 * r.T * c.kv_heads;
  const int64_t per = kThreads / (D / kVec), ctas = (rows + per - 1) / per;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (write)
    kv_write_kernel<T, D, kI8><<<(unsigned)ctas, kThreads, 0, st>>>(
        r.k, r.v, r.k_stride, r.v_stride, r.slots, rows, g, c.k, c.v, c.k_scale, c.v_scale);
  else
    kv_read_kernel<T, D, kI8><<<(unsigned)ctas, kThreads, 0, st>>>(
        c.k, c.v, c.k_scale, c.v_scale, r.slots, rows, g, r.k, r.v, r.k_stride, r.v_stride);
  return cudaGetLastError();
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
