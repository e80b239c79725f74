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
// its whole turns, off by 2^-33 turns at most (by as much again for a frequency of 2^32,
// as 1 / (2 pi) has 96 bits).  With the integer's 2^-33 and fp32's 2^-28: under 2^-27.
//
// head_dim / 8 neighbouring threads have a token and go through its heads, kRows
// rows at a time, the next ones on their way; a thread holds two pieces of four values
// that make four pairs of its own, so neither the rotation nor its loads and stores need
// an exchange, and its cosines and sines are made once.  (A CTA with a table of four
// tokens' angles in shared memory, whose threads took the rows in any order: 67 us for 38
// on 8192 tokens of 40 + 8 heads of 128, 94 for 43 into a bf16 cache, 369 for 154 on 20,011
// of 24 + 4 of 256 into int8 and out again.)  More CTAs an SM, which leave fewer registers,
// lost: 41 us with five of 128 threads, 46 with six.
//
// Measured in CUDA graphs: those 8192 tokens, norms, three axes, bf16 in 39 us (5.2 TB/s,
// 77% of the copy rate), 44 into a bf16 cache with the values (5.3 TB/s); 5003 tokens of 28
// heads of 256, a quarter rotated, fp32 in 48 us (6.0 TB/s); 64 tokens of 48 heads in 3.4 us.
#include <type_traits>

#include "kv_row.cuh"
#include "packed.cuh"

namespace ptq {
namespace {

constexpr int kThreads = 128;
// Rows a thread has in work, and as many on their way.  (8192 tokens of 48 heads of 128, bf16:
// 38 us with four, 50 with two; 5003 of 28 of 256, fp32: 52 and 48.)
template <Act T>
constexpr int kRowsOf = T == Act::F32 ? 2 : 4;

enum Dest { kTensor, kBf16, kI8 };  // where keys go (and values, unless kTensor)

struct Args {
  RopeArgs a;
  CacheGeometry g;  // kBf16, kI8
  int heads, per;   // of a token (q, k and, into a cache, v), of a thread
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

// Cosine and sine of at 2^-32 turns.  The nearest quarter comes off before the angle is rounded to
// fp32, to 2^-28 of a turn then (a half turn's 31 bits rounded to 24 were off by 2^-26).
__device__ __forceinline__ void turn(uint32_t at, float* c, float* s) {
  const uint32_t quarters = (at + (1u << 29)) >> 30;
  float x, y;
  sincospif((float)(int32_t)(at - (quarters << 30)) * 0x1p-31f, &y, &x);
  const float a = quarters & 1 ? y : x, b = quarters & 1 ? x : y;
  *c = (quarters + 1) & 2 ? -a : a;
  *s = quarters & 2 ? -b : b;
}

// Four values as they are in memory, and in fp32.
template <Act T>
using Raw4 = std::conditional_t<T == Act::F32, float4, uint2>;
template <Act T>
__device__ __forceinline__ Raw4<T> load4(const char* p) {
  return *reinterpret_cast<const Raw4<T>*>(p);
}
__device__ __forceinline__ void value4(const float4& a, uint64_t* x) {
  x[0] = pair(a.x, a.y), x[1] = pair(a.z, a.w);
}
__device__ __forceinline__ void value4(const uint2& a, uint64_t* x) {
  x[0] = pair(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u));
  x[1] = pair(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
}
template <Act T>
__device__ __forceinline__ void store4(char* p, const uint64_t* x) {
  float v[4];
  unpair(x[0], v[0], v[1]);
  unpair(x[1], v[2], v[3]);
  if constexpr (T == Act::F32)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) { return v >> 32 | v << 32; }

// A mean of squares in which some that vanished may count, or over the range (or NaN).
constexpr float kLeast = 0x1p-124f;
__device__ __forceinline__ bool is_rare(float mean) {
  return __float_as_uint(mean) - __float_as_uint(kLeast) >= 0x7f800000u - __float_as_uint(kLeast);
}

template <Act T, int D, Dest kDest>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args p) {
  constexpr int kLanes = D / kVec, kGroups = kThreads / kLanes, kSize = T == Act::F32 ? 4 : 2, kRows = kRowsOf<T>;
  constexpr int kOut = kDest == kI8 ? 1 : 2;  // bytes of a cached value
  const RopeArgs& a = p.a;
  const int lane = threadIdx.x % kLanes;
  const int64_t t = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes;
  const bool there = t < a.T;
  const int first = blockIdx.y * p.per, last = min(first + p.per, p.heads);
  pdl_release();
  pdl_wait();
  const int half = a.rotary / 2;
  const bool rotates = 8 * lane < a.rotary;
  // this thread's pieces of a row
  const int e0 = rotates && !a.near ? 4 * lane : 8 * lane, e1 = rotates && !a.near ? half + 4 * lane : 8 * lane + 4;

  // The kinds of heads (0 q, 1 k, 2 v): each one's rows of this thread, one after the other.
  Raw4<T> next[kRows][2];
  auto from_of = [&](int kind) {
    return static_cast<const char*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
           t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) * kSize;
  };
  auto load = [&](const char* row, int n) {  // n rows
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (there && u < n) {
        next[u][0] = load4<T>(row + (u * D + e0) * kSize);
        next[u][1] = load4<T>(row + (u * D + e1) * kSize);
      }
  };
  // kind k has heads [begin(k), begin(k) + count(k)) of this thread's
  auto begin = [&](int k) { return max(first - (k == 0 ? 0 : a.Hq + (k - 1) * a.Hkv), 0); };
  auto end = [&](int k) { return min(last - (k == 0 ? 0 : a.Hq + (k - 1) * a.Hkv), k == 0 ? a.Hq : a.Hkv); };
  int kind = 0;
  while (kind < 3 && begin(kind) >= end(kind)) ++kind;
  if (kind == 3) return;
  load(from_of(kind) + (int64_t)begin(kind) * D * kSize, end(kind) - begin(kind));

  // (cos, cos) and (-sin, sin) of pairs that lie side by side, else pairs of cosines and of sines
  uint64_t c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = pair(1.0f, 1.0f), s[i] = 0;
  if (rotates && first < a.Hq + a.Hkv) {
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = __ldg(a.inv_freq + 4 * lane + i);
      const int ax = a.axis ? __ldg(a.axis + 4 * lane + i) : 0;
      cs[i] = 1.0f, sn[i] = 0.0f;  // a pair of no axis stays as it is
      if ((unsigned)ax < (unsigned)a.axes && there) {
        const int64_t pos = __ldg(a.pos + ax * a.pos_stride + t);
        turn((uint32_t)(((uint64_t)pos * turns_of(f) + (1ull << 31)) >> 32), cs + i, sn + i);
        if (!(fabsf(f) < __int_as_float(0x7f800000))) cs[i] = sn[i] = __int_as_float(0x7fc00000);
      }
    }
    if (a.near) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = pair(cs[i], cs[i]), s[i] = pair(-sn[i], sn[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) c[i] = pair(cs[2 * i], cs[2 * i + 1]), s[i] = pair(sn[2 * i], sn[2 * i + 1]);
    }
  }

#pragma unroll 1
  for (; kind < 3; ++kind) {
    const int h0 = begin(kind), h1 = end(kind);
    if (h0 >= h1) continue;
    const float* gain = kind == 0 ? a.q_gain : kind == 1 ? a.k_gain : nullptr;
    uint64_t g[4] = {};
    if (gain) {
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain + e0)),
                   g1 = __ldg(reinterpret_cast<const float4*>(gain + e1));
      value4(g0, g), value4(g1, g + 2);
    }
    // where rows go: a tensor, or this token's place in the cache
    const bool cached = kDest != kTensor && kind > 0;
    char* to;
    int64_t step = (int64_t)D * kSize, row = 0;
    bool stored = there;
    if (cached) {
      const int slot = there ? __ldg(a.slots + t) : -1;
      stored = (unsigned)slot < (unsigned)p.g.pages_slots;
      row = cache_row(stored ? slot : 0, 0, p.g);
      to = static_cast<char*>(kind == 1 ? a.ck : a.cv) + row * (D * kOut);
      step = (int64_t)p.g.page_tokens.d * (D * kOut);
    } else {
      to = static_cast<char*>(kind == 0 ? a.q_out : a.k_out) + t * (kind == 0 ? a.qo_stride : a.ko_stride) * kSize;
    }
    const char* from = from_of(kind);
#pragma unroll 1
    for (int h = h0; h < h1; h += kRows) {
      uint64_t x[kRows][4];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0;
        if (there && h + u < h1) value4(next[u][0], x[u]), value4(next[u][1], x[u] + 2);
      }
      // the next rows, of this kind or the one after
      if (h + kRows < h1) {
        load(from + (int64_t)(h + kRows) * D * kSize, h1 - h - kRows);
      } else {
        int k = kind + 1;
        while (k < 3 && begin(k) >= end(k)) ++k;
        if (k < 3) load(from_of(k) + (int64_t)begin(k) * D * kSize, end(k) - begin(k));
      }
      if (gain) {
        float ss[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          uint64_t q = mul2(x[u][0], x[u][0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) q = fma2(x[u][i], x[u][i], q);
          float lo, hi;
          unpair(q, lo, hi);
          ss[u] = lo + hi;
        }
#pragma unroll
        for (int i = kLanes / 2; i > 0; i >>= 1)
#pragma unroll
          for (int u = 0; u < kRows; ++u) ss[u] += __shfl_xor_sync(~0u, ss[u], i);
        float inv[kRows];
        bool any = false;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          ss[u] = ss[u] * (1.0f / D) + a.eps;
          inv[u] = rsqrtf(ss[u]);
          any |= is_rare(ss[u]);
        }
        if (__builtin_expect(__any_sync(~0u, any), 0)) {
#pragma unroll
          for (int u = 0; u < kRows; ++u) {
            // again over a power of two
            const bool small = ss[u] < kLeast;
            const float by = small ? 0x1p96f : 0x1p-70f;
            float m = 0.0f, v[kVec], s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) unpair(x[u][i], v[2 * i], v[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) m = fmaxf(m, fabsf(v[i])), s2 = fmaf(v[i] * by, v[i] * by, s2);
#pragma unroll
            for (int i = kLanes / 2; i > 0; i >>= 1) {
              m = fmaxf(m, __shfl_xor_sync(~0u, m, i));
              s2 += __shfl_xor_sync(~0u, s2, i);
            }
            if (is_rare(ss[u]) && m < __int_as_float(0x7f800000)) {
              // x by (1 / root) by the power or the other way round: no product loses bits
              const float of = rsqrtf(s2 * (1.0f / D) + a.eps * by * by);
              inv[u] = small ? of : by;
#pragma unroll
              for (int i = 0; i < 4; ++i) x[u][i] = mul2(x[u][i], small ? pair(by, by) : pair(of, of));
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const uint64_t ii = pair(inv[u], inv[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[u][i] = mul2(mul2(x[u][i], ii), g[i]);
        }
      }
      if (rotates && kind < 2) {
        if (a.near) {
#pragma unroll
          for (int u = 0; u < kRows; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = fma2(x[u][i], c[i], mul2(swapped(x[u][i]), s[i]));
        } else {
#pragma unroll
          for (int u = 0; u < kRows; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint64_t xa = x[u][i], xb = x[u][2 + i];
              x[u][i] = fma2(xa, c[i], mul2(xb, s[i] ^ 0x8000000080000000ull));
              x[u][2 + i] = fma2(xb, c[i], mul2(xa, s[i]));
            }
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        char* at = to + (h + u) * step;
        const bool ok = stored && h + u < h1;
        if (!cached) {
          if (ok) {
            store4<T>(at + e0 * kSize, x[u]);
            store4<T>(at + e1 * kSize, x[u] + 2);
          }
        } else if constexpr (kDest == kBf16) {
          if (ok) {
            store4<Act::BF16>(at + e0 * 2, x[u]);
            store4<Act::BF16>(at + e1 * 2, x[u] + 2);
          }
        } else if constexpr (kDest == kI8) {
          float v[kVec];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpair(x[u][i], v[2 * i], v[2 * i + 1]);
          uint32_t code[2];
          const float sc = quantise<kLanes, true, true>(v, code);
          if (ok) {
            *reinterpret_cast<uint32_t*>(at + e0) = code[0];
            *reinterpret_cast<uint32_t*>(at + e1) = code[1];
            if (lane == 0) (kind == 2 ? a.vs : a.ks)[row + (int64_t)(h + u) * p.g.page_tokens.d] = sc;
          }
        }
      }
    }
  }
}

template <Act T, int D, Dest kDest>
cudaError_t launch(const RopeArgs& a, const ptq_kv_cache* c, cudaStream_t st) {
  constexpr int kGroups = kThreads / (D / kVec), kRows = kRowsOf<T>;
  const int64_t heads = a.Hq + a.Hkv * (kDest == kTensor ? 1 : 2);
  // A thread goes through all heads of its token, or, where that leaves SMs without work,
  // through as many as keep them busy, kRows at least.
  const int64_t x = (a.T + kGroups - 1) / kGroups, most = (heads + kRows - 1) / kRows;
  int64_t y = (4 * 152 + x - 1) / x;
  y = y < most ? y : most;
  const int64_t per = ((heads + y - 1) / y + kRows - 1) / kRows * kRows;
  y = (heads + per - 1) / per;
  if (x > INT32_MAX || y > 65535) return cudaErrorInvalidValue;
  const Args p{a, CacheGeometry{c ? (int)(c->pages * c->page_tokens) : 0, Divider(c ? c->page_tokens : 1),
                                Divider(c ? c->kv_heads : 1)},
               (int)heads, (int)per};
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
