// k_rope.cu -- norms of queries and keys for each head and their position
// rotation in one pass, into tensors or on the way into a paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * g,
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//   t = pos[axis of the pair] * inv_freq[pair]
//
// One read and one write of each value: HBM bounds it on prompts, the launch
// and a chain of latencies (position, angle, row) at a decode step.  fp32
// throughout, one rounding at the end; int8 rows are quantised from the rotated
// fp32 values.
//
// Angles.  Positions go far (2^31), and an fp32 product pos * inv_freq is off
// by 2^-24 of the angle: 0.03 at 2^19.  A frequency is made a 64-bit fraction
// of a turn, inv_freq / (2 pi) modulo 1, by integer products (fp64 runs at two
// operations a clock and SM); pos times that, modulo 2^64, is the angle without
// its whole turns, off by 2^-33 turns at most.
//
// A CTA has a few tokens: its threads make their cosines and sines once, in
// shared memory, for all heads.  Then head_dim / 8 neighbouring threads hold a
// row, each two pieces of four values that make four pairs, so neither the
// rotation nor its loads and stores need an exchange; the rows of kRows heads
// are loaded together.
#include "kv_row.cuh"

namespace ptq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;      // rows a thread has in flight
constexpr int kTokens = 4;    // most tokens of a CTA
constexpr int kMaxPairs = 128;

enum Dest { kTensor, kBf16, kI8 };  // where keys go (and values, unless kTensor)

struct Args {
  RopeArgs a;
  CacheGeometry g;       // kBf16, kI8
  int heads;             // of a token: q, k and, into a cache, v
  int tokens, per;       // of a CTA: tokens, heads
  Divider by_per, by_half;
};

// f / (2 pi) modulo 1, times 2^64: f is m 2^e with m a 24-bit integer, and m
// floor(2^96 / (2 pi)) has 118 bits.
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t b = __float_as_uint(f), ex = b >> 23 & 0xff;
  const uint32_t m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int shift = 32 + 150 - (int)(ex ? ex : 1);  // the product's units are 2^(e - 96)
  const uint64_t lo = (uint64_t)m * 0x7f09d5f4u, mid = (uint64_t)m * 0x9391054au + (lo >> 32),
                 hi = (uint64_t)m * 0x28be60dbu + (mid >> 32);
  const unsigned __int128 p = (unsigned __int128)hi << 64 | (mid & 0xffffffffu) << 32 | (uint32_t)lo;
  const uint64_t t = shift >= 128 ? 0 : shift >= 0 ? (uint64_t)(p >> shift)
                                    : shift > -64 ? (uint64_t)p << -shift : 0;
  return b >> 31 ? 0 - t : t;
}

template <Act T>
__device__ __forceinline__ void load4(const void* p, int64_t e, float* x) {
  if constexpr (T == Act::F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + e);
    x[0] = __uint_as_float(a.x << 16), x[1] = __uint_as_float(a.x & 0xffff0000u);
    x[2] = __uint_as_float(a.y << 16), x[3] = __uint_as_float(a.y & 0xffff0000u);
  }
}
template <Act T>
__device__ __forceinline__ void store4(void* p, int64_t e, const float* x) {
  if constexpr (T == Act::F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + e) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + e) =
        make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}

template <Act T, int D, Dest kDest>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args p) {
  constexpr int kLanes = D / kVec, kGroups = kThreads / kLanes;
  __shared__ __align__(16) float2 turn[kTokens * kMaxPairs];  // (cos, sin)
  const RopeArgs& a = p.a;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  pdl_release();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int n_tok = (int)min((int64_t)p.tokens, a.T - t0), h0 = blockIdx.y * p.per;
  const int rows = n_tok * p.per, half = a.rotary / 2;
  const bool rotates = 8 * lane < a.rotary;
  // this thread's pieces of a row
  const int e0 = rotates && !a.near ? 4 * lane : 8 * lane, e1 = rotates && !a.near ? half + 4 * lane : 8 * lane + 4;

  struct Row {
    int64_t t;
    int in_cta, h;  // token of the CTA, head among q, k, v
    bool there;
  };
  auto row_at = [&](int r) {
    Row w;
    w.in_cta = p.by_per(r);
    w.h = h0 + r - w.in_cta * p.per;
    w.t = t0 + w.in_cta;
    w.there = r < rows && w.h < p.heads;
    return w;
  };
  float x[kRows][kVec];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const Row w = row_at(r0 + u * kGroups);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[u][i] = 0.0f;
      if (!w.there) continue;
      const int hk = w.h - a.Hq, hv = hk - a.Hkv;
      const void* from = hk < 0 ? a.q : hv < 0 ? a.k : a.v;
      const int64_t e = w.t * (hk < 0 ? a.q_stride : hv < 0 ? a.k_stride : a.v_stride) +
                        (int64_t)(hk < 0 ? w.h : hv < 0 ? hk : hv) * D;
      load4<T>(from, e + e0, x[u]);
      load4<T>(from, e + e1, x[u] + 4);
    }
  };
  load(group);
  for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
    const int tok = p.by_half(i), pair = i - tok * half;
    const float f = __ldg(a.inv_freq + pair);
    const int ax = a.axis ? __ldg(a.axis + pair) : 0;
    float2 cs = make_float2(1.0f, 0.0f);  // a pair of no axis stays as it is
    if ((unsigned)ax < (unsigned)a.axes) {
      const int64_t pos = __ldg(a.pos + ax * a.pos_stride + t0 + tok);
      const uint64_t at = (uint64_t)pos * turns_of(f) + (1ull << 31);
      sincospif((float)(int32_t)(at >> 32) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31 half turns
      if (!(fabsf(f) < __int_as_float(0x7f800000))) cs.x = cs.y = __int_as_float(0x7fc00000);
    }
    turn[i] = cs;
  }
  __syncthreads();

#pragma unroll 1
  for (int r0 = group; r0 - group < rows; r0 += kRows * kGroups) {
    if (r0 != group) load(r0);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const Row w = row_at(r0 + u * kGroups);
      const int hk = w.h - a.Hq, hv = hk - a.Hkv;
      const bool value = kDest != kTensor && hv >= 0;
      const float* gain = value ? nullptr : hk < 0 ? a.q_gain : a.k_gain;
      if (a.q_gain || a.k_gain) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
        for (int i = kLanes / 2; i > 0; i >>= 1) ss += __shfl_xor_sync(~0u, ss, i);
        if (__builtin_expect(__any_sync(~0u, !(ss < __int_as_float(0x7f800000))), 0)) {
          // the squares of a row of finite values overflow: over a power of two
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) m = fmaxf(m, fabsf(x[u][i]));
#pragma unroll
          for (int i = kLanes / 2; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, i));
          const bool over = !(ss < __int_as_float(0x7f800000)) && gain && m < __int_as_float(0x7f800000);
          float s2 = 0.0f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const float y = x[u][i] * 0x1p-96f;
            s2 = fmaf(y, y, s2);
            if (over) x[u][i] = y;
          }
#pragma unroll
          for (int i = kLanes / 2; i > 0; i >>= 1) s2 += __shfl_xor_sync(~0u, s2, i);
          if (over) ss = s2;  // (eps is far below a unit of it)
        }
        if (gain) {
          const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
          const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain + e0)),
                       g1 = __ldg(reinterpret_cast<const float4*>(gain + e1));
          const float g[kVec] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
          for (int i = 0; i < kVec; ++i) x[u][i] = x[u][i] * inv * g[i];
        }
      }
      if (rotates && !value && w.there) {
        const float4* cs = reinterpret_cast<const float4*>(turn + w.in_cta * half + 4 * lane);
        const float4 c01 = cs[0], c23 = cs[1];
        const float c[4] = {c01.x, c01.z, c23.x, c23.z}, s[4] = {c01.y, c01.w, c23.y, c23.w};
        auto turned = [&](float& ya, float& yb, int i) {
          const float xa = ya, xb = yb;
          ya = xa * c[i] - xb * s[i];
          yb = xb * c[i] + xa * s[i];
        };
        if (a.near) {
#pragma unroll
          for (int i = 0; i < 4; ++i) turned(x[u][2 * i], x[u][2 * i + 1], i);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) turned(x[u][i], x[u][4 + i], i);
        }
      }
      if (kDest == kTensor || hk < 0) {
        if (w.there && hk < 0) {
          const int64_t e = w.t * a.qo_stride + (int64_t)w.h * D;
          store4<T>(a.q_out, e + e0, x[u]);
          store4<T>(a.q_out, e + e1, x[u] + 4);
        } else if (w.there) {
          const int64_t e = w.t * a.ko_stride + (int64_t)hk * D;
          store4<T>(a.k_out, e + e0, x[u]);
          store4<T>(a.k_out, e + e1, x[u] + 4);
        }
      }
      if constexpr (kDest != kTensor) {
        const int slot = w.there && hk >= 0 ? __ldg(a.slots + w.t) : -1;
        const bool ok = (unsigned)slot < (unsigned)p.g.pages_slots;
        const int64_t row = ok ? cache_row(slot, value ? hv : hk, p.g) : 0;
        if constexpr (kDest == kBf16) {
          if (ok) {
            void* to = value ? a.cv : a.ck;
            store4<Act::BF16>(to, row * D + e0, x[u]);
            store4<Act::BF16>(to, row * D + e1, x[u] + 4);
          }
        } else {
          uint32_t code[2];
          const float s = quantise<kLanes, true>(x[u], code);
          if (ok) {
            char* to = static_cast<char*>(value ? a.cv : a.ck) + row * D;
            *reinterpret_cast<uint32_t*>(to + e0) = code[0];
            *reinterpret_cast<uint32_t*>(to + e1) = code[1];
            if (lane == 0) (value ? a.vs : a.ks)[row] = s;
          }
        }
      }
    }
  }
}

template <Act T, int D, Dest kDest>
cudaError_t launch(const RopeArgs& a, const ptq_kv_cache* c, cudaStream_t st) {
  constexpr int kGroups = kThreads / (D / kVec);
  const int64_t heads = a.Hq + a.Hkv * (kDest == kTensor ? 1 : 2);
  // Few tokens: a row a thread group, over as many CTAs as that takes.  Many: a
  // CTA has all heads of kTokens tokens, whose angles are made once.
  const bool many = a.T >= 1024;
  const int64_t per = many || heads <= kGroups ? heads : kGroups;
  const int64_t tokens = many ? kTokens : 1;
  const int64_t x = (a.T + tokens - 1) / tokens, y = (heads + per - 1) / per;
  if (x > INT32_MAX || y > 65535 || per > INT32_MAX / kTokens) return cudaErrorInvalidValue;
  const Args p{a, CacheGeometry{c ? (int)(c->pages * c->page_tokens) : 0, Divider(c ? c->page_tokens : 1),
                                Divider(c ? c->kv_heads : 1)},
               (int)heads, (int)tokens, (int)per, Divider(per), Divider(a.rotary ? a.rotary / 2 : 1)};
  return launch_pdl(rope_kernel<T, D, kDest>, dim3((unsigned)x, (unsigned)y), dim3(kThreads), 0, st, p);
}

template <Act T, Dest kDest>
cudaError_t by_dim(const RopeArgs& a, const ptq_kv_cache* c, int64_t D, cudaStream_t st) {
  switch (D) {
    case 64: return launch<T, 64, kDest>(a, c, st);
    case 128: return launch<T, 128, kDest>(a, c, st);
    default: return launch<T, 256, kDest>(a, c, st);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, const ptq_kv_cache* c, int64_t D, cudaStream_t st) {
  const bool f32 = a.t == Act::F32;
  if (!c) return f32 ? by_dim<Act::F32, kTensor>(a, c, D, st) : by_dim<Act::BF16, kTensor>(a, c, D, st);
  if (c->type == PTQ_KV_I8)
    return f32 ? by_dim<Act::F32, kI8>(a, c, D, st) : by_dim<Act::BF16, kI8>(a, c, D, st);
  return f32 ? by_dim<Act::F32, kBf16>(a, c, D, st) : by_dim<Act::BF16, kBf16>(a, c, D, st);
}

}  // namespace ptq
