// k_attn_prefill.cu -- attention of packed prompts on the 5th-generation
// tensor cores.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - m),  O = P V,  out = O / sum P
//
// 4 head_dim operations a visible (query, key) pair and query head against
// one exponential: the tensor cores bound it, the exponentials at head_dim
// 64.
//
// Tile.  128 rows of Q are tpt tokens of hg query heads that share a kv head
// (row = token * hg + head, one TMA box), against tiles of 128 keys.  S and O
// live in TMEM; P goes back there as bf16 over S's columns and is the A
// operand of the second product, so only K and V pass through shared memory.
// A CTA holds two Q tiles (head_dim up to 128), neighbours in the sequence,
// that share each K and V tile; at head_dim 256 one Q tile whose S has two
// buffers.  Either way the tensor core always has the other S in work while
// the softmax of one runs:
//     QK(0) QK(1) PV(0) QK(2) PV(1) QK(3) PV(2) ...
// and because the tensor core runs in order, PV(i) having been issued before
// QK(i + 2) is all that keeps a slot's P from being overwritten.
//
// Warps: four for the softmax of each Q tile (a thread holds a row: its
// maximum and sum need no shuffle), one that issues the TMA loads, one that
// issues the MMAs.  The maximum that P refers to moves only when a row's
// grows by more than 2^8 over it: P up to 2^8 costs fp32 sums nothing, and
// rescaling O (TMEM to registers and back) becomes rare.
//
// A key that a row does not see has P = 0, and 0 times a non-finite value is
// NaN: rows whose output is not finite though their sum is are computed again
// one by one over the keys they see.
//
// Every wait is bounded; one that runs out raises the device status word and
// the CTA drains what it has in flight and exits.
#include <cuda_bf16.h>

#include "async_util.cuh"
#include "attn_row.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kRows = 128;  // rows of a Q tile
constexpr int kKeys = 128;  // keys of a K and V tile
constexpr float kSlack = 8.0f;  // log2 of the largest P

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;    // Q tiles of a CTA
  static constexpr int kCols = D < 128 ? D : 128;    // columns of a ring unit
  static constexpr int kUnits = D / kCols;           // units of a K or V tile
  static constexpr int kUnit = kKeys * kCols * 2;    // bytes
  static constexpr int kRing = D == 64 ? 8 : 5;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSoftmax = 4 * kTiles;        // softmax warps
  static constexpr int kThreads = 32 * (kSoftmax + 2);
  static constexpr int kOffRing = kTiles * kQ;
  static constexpr int kOffBar = kOffRing + kRing * kUnit;
  // full[kRing] empty[kRing] q s[2] p[2] o[2] pv done
  static constexpr int kBars = 2 * kRing + 1 + 2 + 2 + 2 + 1 + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 64;
};
static_assert(Cfg<128>::kSmem <= 227 * 1024 && Cfg<256>::kSmem <= 227 * 1024, "shared memory");

struct Args {
  PrefillArgs a;
  int G, hg, tpt;  // query heads of a kv head; heads and tokens of a Q tile
};

__device__ __forceinline__ int clamped(int v, int64_t hi) {
  return v < 0 ? 0 : v > hi ? (int)hi : v;
}

struct Span {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Span span_of(const PrefillArgs& a, int b) {
  const int q0 = clamped(__ldg(a.cu_q + b), a.Tq), q1 = clamped(__ldg(a.cu_q + b + 1), a.Tq);
  const int k0 = clamped(__ldg(a.cu_k + b), a.Tk), k1 = clamped(__ldg(a.cu_k + b + 1), a.Tk);
  return {q0, max(0, q1 - q0), k0, max(0, k1 - k0)};
}

template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float((uint32_t)__ldg(p + i) << 16);
}

// One query row by a warp: query t (of all), head hq, over keys [k0, end).
template <int D>
__device__ __noinline__ void attend_row(const PrefillArgs& a, int t, int hq, int h, int k0, int end) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  float q[N];
  load_bf16(a.q + (int64_t)t * a.q_stride + (int64_t)hq * D + lane * N, q);
  RowState<D> r;
  for (int j = k0; j < end; ++j) {
    float k[N], v[N];
    load_bf16(a.k + (int64_t)j * a.k_stride + (int64_t)h * D + lane * N, k);
    load_bf16(a.v + (int64_t)j * a.v_stride + (int64_t)h * D + lane * N, v);
    r.add(q, k, v, a.scale * kLog2e);
  }
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;
#pragma unroll
  for (int i = 0; i < N; ++i)
    a.out[((int64_t)t * a.Hq + hq) * D + lane * N + i] =
        __bfloat16_as_ushort(__float2bfloat16_rn(r.o[i] * inv));
}

// ---- tensor core -------------------------------------------------------------------

// Shared-memory descriptor of a 128-byte-swizzled tile: 8-row atoms 1024
// bytes apart; lead: bytes between column blocks of 64 (N-major operands).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 sums, A and B bf16, M = 128; bit 16: B is
// N-major (V, whose rows are keys).
template <int N, bool kNMajor>
__device__ __forceinline__ constexpr uint32_t idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | (kNMajor ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

#define PTQ_R8(v, i) \
  "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
      "=r"(v[i + 6]), "=r"(v[i + 7])
#define PTQ_W8(v, i) \
  "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
      "r"(v[i + 6]), "r"(v[i + 7])

// 32 columns of this warp's 32 TMEM lanes, a row for each lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : PTQ_R8(v, 0), PTQ_R8(v, 8), PTQ_R8(v, 16), PTQ_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(addr),
      PTQ_W8(v, 0), PTQ_W8(v, 8), PTQ_W8(v, 16), PTQ_W8(v, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---- the order of the work -----------------------------------------------------------
// Work item i of a head: sequences are cut into runs of `run` queries, the
// runs that come late in their sequence (under a causal mask those with the
// most keys) first.  With f(t) = sum over sequences of max(0, runs - t), the
// items of run number t are [f(t + 1), f(t)).  One warp; false: no such item.
__device__ bool find_item(const PrefillArgs& a, int run, int64_t i, int* b_out, int* t_out) {
  const int lane = threadIdx.x & 31;
  auto runs = [&](int64_t b) { return b < a.B ? (span_of(a, (int)b).nq + run - 1) / run : 0; };
  int most = 0;
  const int first = runs(lane);
  for (int64_t b = lane; b < a.B; b += 32) most = max(most, runs(b));
  most = __reduce_max_sync(~0u, most);
  auto f = [&](int t) {
    int64_t n = max(0, first - t);
    for (int64_t b = lane + 32; b < a.B; b += 32) n += max(0, runs(b) - t);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) n += __shfl_xor_sync(~0u, n, s);
    return n;
  };
  if (f(0) <= i) return false;
  int lo = 0, hi = most;  // f(lo) > i >= f(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (f(mid) > i)
      lo = mid;
    else
      hi = mid;
  }
  int64_t rank = i - f(lo + 1);  // among the sequences with more than lo runs
  for (int64_t b0 = 0; b0 < a.B; b0 += 32) {
    const unsigned has = __ballot_sync(~0u, runs(b0 + lane) > lo);
    const int n = __popc(has);
    if (rank < n) {
      *b_out = (int)b0 + __fns(has, 0, (int)rank + 1);
      *t_out = lo;
      return true;
    }
    rank -= n;
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args p,
                        int* status) {
  using C = Cfg<D>;
  constexpr int kTiles = C::kTiles;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *full = bars, *empty = bars + C::kRing, *q_full = bars + 2 * C::kRing;
  uint64_t *s_full = q_full + 1, *p_full = s_full + 2, *o_full = p_full + 2, *pv_done = o_full + 2,
           *all_done = pv_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* item = reinterpret_cast<int*>(smem + C::kOffMisc + 8);  // sequence (-1: none), run

  const PrefillArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kLoad = C::kSoftmax, kMma = C::kSoftmax + 1;

  pdl_release();
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kLoad) {
    if (lane == 0) {
      for (int i = 0; i < C::kRing; ++i) {
        mbar_init(full + i, 1);
        mbar_init(empty + i, 1);
      }
      mbar_init(q_full, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(s_full + i, 1);
        mbar_init(p_full + i, 4);  // the four softmax warps of a tile
        mbar_init(o_full + i, 1);
      }
      mbar_init(pv_done, 1);
      mbar_init(all_done, 1);
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  } else if (warp == 0) {
    pdl_wait();
    int b = -1, t = 0;
    if (!find_item(a, kTiles * p.tpt, blockIdx.x, &b, &t)) b = -1;
    if (lane == 0) {
      item[0] = b;
      item[1] = t;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const int b = item[0];
  if (b >= 0) {
    const Span sp = span_of(a, b);
    const int blocks = p.G / p.hg;  // head blocks of a kv head
    const int h = blockIdx.y / blocks, hq0 = h * p.G + (blockIdx.y % blocks) * p.hg;
    // Q tile s: queries tok(s) .. tok(s) + tpt - 1 of the sequence; keys of its
    // last query; K tiles
    int first[kTiles], n[kTiles];
#pragma unroll
    for (int s = 0; s < kTiles; ++s) {
      first[s] = (item[1] * kTiles + s) * p.tpt;
      const int last = min(first[s] + p.tpt, sp.nq) - 1;
      const int keys = a.causal ? min(sp.nk, sp.nk - sp.nq + last + 1) : sp.nk;
      n[s] = first[s] < sp.nq && keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
    }
    int most = n[0];
    if (kTiles == 2) most = max(most, n[kTiles - 1]);
    const uint32_t ring = smem_addr(smem + C::kOffRing), qs = smem_addr(smem);
    bool ok = true;

    if (warp == kLoad) {
      // ---- loads: Q, then K_0 V_0 K_1 V_1 ... through the ring ----------------------
      if (lane == 0 && most > 0) {
        const int rows = p.hg * p.tpt;
        int tiles = 0;
        for (int s = 0; s < kTiles; ++s) tiles += n[s] > 0;
        mbar_expect_tx(q_full, (uint32_t)(tiles * rows * D * 2));
        for (int s = 0; s < kTiles; ++s)
          if (n[s] > 0)
            for (int c = 0; c < D / 64; ++c)
              tma_3d(qs + s * C::kQ + c * kRows * 128, &map_q, 64 * c, hq0, sp.q0 + first[s], q_full);
        int u = 0;  // units issued
        for (int j = 0; j < most && ok; ++j)
          for (int kv = 0; kv < 2 && ok; ++kv)
            for (int i = 0; i < C::kUnits && ok; ++i, ++u) {
              const int st = u % C::kRing, round = u / C::kRing;
              if (round > 0) ok = mbar_wait(empty + st, (round - 1) & 1, abort_flag);
              if (!ok) break;
              mbar_expect_tx(full + st, C::kUnit);
              for (int c = 0; c < C::kCols / 64; ++c)
                tma_3d(ring + st * C::kUnit + c * kKeys * 128, kv ? &map_v : &map_k,
                       i * C::kCols + 64 * c, h, sp.k0 + j * kKeys, full + st);
            }
        // whatever becomes of the MMAs, the copies land before the CTA ends
        for (int v = max(0, u - C::kRing); v < u; ++v)
          static_cast<void>(mbar_wait(full + v % C::kRing, (v / C::kRing) & 1, nullptr));
        static_cast<void>(mbar_wait(q_full, 0, nullptr));
      }
    } else if (warp == kMma) {
      // ---- MMAs ------------------------------------------------------------------------
      if (lane == 0) {
        struct Item {
          int j, s;
        };
        auto valid = [&](Item i) { return i.j < most; };
        auto next = [&](Item i) {
          if constexpr (kTiles == 1) {
            ++i.j;
          } else {
            do {
              i = i.s == 0 ? Item{i.j, 1} : Item{i.j + 1, 0};
            } while (i.j < most && i.j >= n[i.s]);
          }
          return i;
        };
        auto slot_of = [&](Item i) { return kTiles == 1 ? i.j & 1 : i.s; };
        auto use_of = [&](Item i) { return kTiles == 1 ? i.j >> 1 : i.j; };
        auto last_user = [&](Item i) {
          return kTiles == 1 || i.s == 1 || i.j >= n[kTiles - 1];
        };
        auto qk = [&](Item i) {
          const uint32_t d = tmem + slot_of(i) * kKeys;
          for (int k = 0; k < C::kUnits && ok; ++k) {
            const int u = 2 * i.j * C::kUnits + k, st = u % C::kRing;
            ok = mbar_wait(full + st, (u / C::kRing) & 1, abort_flag);
            if (!ok) return;
            fence_after();
#pragma unroll
            for (int c = 0; c < C::kCols / 64; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_ss(d, tile_desc(qs + i.s * C::kQ + (k * (C::kCols / 64) + c) * kRows * 128 + 32 * e, 16),
                       tile_desc(ring + st * C::kUnit + c * kKeys * 128 + 32 * e, 16),
                       idesc<kKeys, false>(), (k | c | e) != 0);
            if (last_user(i)) mma_commit(empty + st);
          }
          mma_commit(s_full + slot_of(i));
        };
        auto pv = [&](Item i) {
          ok = mbar_wait(p_full + slot_of(i), use_of(i) & 1, abort_flag);
          if (!ok) return;
          fence_after();
          const uint32_t pa = tmem + slot_of(i) * kKeys;
          for (int k = 0; k < C::kUnits && ok; ++k) {
            const int u = (2 * i.j + 1) * C::kUnits + k, st = u % C::kRing;
            ok = mbar_wait(full + st, (u / C::kRing) & 1, abort_flag);
            if (!ok) return;
            fence_after();
            const uint32_t d = tmem + 2 * kKeys + i.s * D + k * C::kCols;
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              mma_ts(d, pa + 8 * e, tile_desc(ring + st * C::kUnit + 2048 * e, kKeys * 128),
                     idesc<C::kCols, true>(), i.j > 0 || e > 0);
            if (last_user(i)) mma_commit(empty + st);
          }
          if constexpr (kTiles == 1) mma_commit(pv_done);
          if (i.j == n[i.s] - 1) mma_commit(o_full + i.s);
        };
        Item i{0, 0};
        if (most > 0) {
          ok = mbar_wait(q_full, 0, abort_flag);
          if (n[0] == 0) i = next(i);
          if (ok) qk(i);
          while (ok && valid(i)) {
            const Item nx = next(i);
            const bool apart = valid(nx) && slot_of(nx) != slot_of(i);
            if (apart) qk(nx);
            if (ok) pv(i);
            if (ok && valid(nx) && !apart) qk(nx);
            i = nx;
          }
        }
        mma_commit(all_done);
      }
    } else {
      // ---- softmax: thread = row of Q tile s ----------------------------------------
      const int s = kTiles == 1 ? 0 : warp >> 2, quarter = warp & 3;
      const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
      const int row = 32 * quarter + lane, tok = first[s] + row / p.hg;
      const bool mine = row < p.hg * p.tpt && tok < sp.nq;
      // keys this row sees, and those its tile's first row sees
      const int sees = a.causal ? min(sp.nk, sp.nk - sp.nq + tok + 1) : sp.nk;
      const int all_see = a.causal ? min(sp.nk, sp.nk - sp.nq + first[s] + 1) : sp.nk;
      const float scale2 = a.scale * kLog2e;
      const uint32_t o_at = tmem + lanes + 2 * kKeys + s * D;
      float m = kNegInf;  // what P refers to, in units of log2
      uint64_t sum2 = pair(0.0f, 0.0f);
      for (int j = 0; j < n[s] && ok; ++j) {
        const int slot = kTiles == 1 ? j & 1 : s, use = kTiles == 1 ? j >> 1 : j;
        const uint32_t at = tmem + lanes + slot * kKeys;
        ok = __all_sync(~0u, mbar_wait(s_full + slot, use & 1, abort_flag));
        if (!ok) break;
        fence_after();
        uint32_t v[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(at + c, v + c);
        tmem_wait_ld();
        if ((j + 1) * kKeys > all_see) {
          const int left = sees - j * kKeys;
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c >= left) v[c] = 0xff800000u;
        }
        float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int c = 0; c < kKeys; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top[e] = fmaxf(top[e], fmaxf(__uint_as_float(v[c + 2 * e]), __uint_as_float(v[c + 2 * e + 1])));
        const float t2 = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale2;
        if (j == 0) {
          m = t2;
        } else if (__any_sync(~0u, t2 > m + kSlack)) {
          // O moves to the new maximum; the product before the last of this
          // tile's has been waited for with S (one Q tile: here)
          const float mn = t2 > m + kSlack ? t2 : m;
          const float f = m == kNegInf ? 0.0f : exp2_fast(m - mn);
          m = mn;
          if constexpr (kTiles == 1) {
            ok = __all_sync(~0u, mbar_wait(pv_done, (j - 1) & 1, abort_flag));
            if (!ok) break;
            fence_after();
          }
          float lo, hi;
          unpair(sum2, lo, hi);
          sum2 = pair(lo * f, hi * f);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_at + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_at + c, o);
          }
        }
        const float z = m == kNegInf ? 0.0f : -m;
        const uint64_t zz = pair(z, z), ss = pair(scale2, scale2);
#pragma unroll
        for (int c = 0; c < kKeys; c += 64) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            unpair(fma2(pair(__uint_as_float(v[c + 2 * e]), __uint_as_float(v[c + 2 * e + 1])), ss, zz), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum2 = add2(sum2, pair(x0, x1));
            w[e] = bf16x2(x0, x1);
          }
          tmem_st32(at + c / 2, w);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + slot);
      }

      // ---- epilogue ----------------------------------------------------------------
      float lo, hi;
      unpair(sum2, lo, hi);
      const float l = lo + hi;
      const int64_t tq = sp.q0 + tok;
      const int hq = hq0 + row % p.hg;
      const bool keys = n[s] > 0;
      if (ok && keys) ok = __all_sync(~0u, mbar_wait(o_full + s, 0, abort_flag));
      if (ok && first[s] < sp.nq) {
        fence_after();
        if (mine && a.lse) a.lse[tq * a.Hq + hq] = l == 0.0f ? kNegInf : m * kLn2 + logf(l);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        // rows go through the dead Q tile so that a row's bytes are stored together
        unsigned char* stage = smem + s * C::kQ + row * 128;
        bool bad = false;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32], w[16];
          if (keys) {
            tmem_ld32(o_at + c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0 = __uint_as_float(o[e]), x1 = __uint_as_float(o[e + 1]);
            if (l == 0.0f) x0 = x1 = 0.0f;
            bad |= !(fabsf(x0) <= 3.4028235e38f) | !(fabsf(x1) <= 3.4028235e38f);
            w[e / 2] = bf16x2(x0 * inv, x1 * inv);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(stage + (c / 64) * kRows * 128 +
                                      ((((c % 64) / 8 + e) ^ (row & 7)) << 4)) =
                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
        __syncwarp();
        constexpr int kPieces = D / 8;  // 16-byte pieces of a row
#pragma unroll 4
        for (int i = lane; i < 32 * kPieces; i += 32) {
          const int r = 32 * quarter + i / kPieces, piece = i % kPieces;
          const int tr = first[s] + r / p.hg;
          if (r < p.hg * p.tpt && tr < sp.nq)
            *reinterpret_cast<uint4*>(a.out + ((int64_t)(sp.q0 + tr) * a.Hq + hq0 + r % p.hg) * D +
                                      8 * piece) =
                *reinterpret_cast<const uint4*>(smem + s * C::kQ + (piece / 8) * kRows * 128 + r * 128 +
                                                (((piece % 8) ^ (r & 7)) << 4));
        }
        // rows whose sum is finite and whose output is not
        unsigned again = __ballot_sync(~0u, mine && bad && l == l);
        while (again) {
          const int who = __ffs(again) - 1;
          again &= again - 1;
          __syncwarp();
          attend_row<D>(a, __shfl_sync(~0u, (int)tq, who), __shfl_sync(~0u, hq, who), h, sp.k0,
                        sp.k0 + __shfl_sync(~0u, sees, who));
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(status, kDevTimeout);
    }
    if (*abort_flag && warp == kMma && lane == 0) static_cast<void>(mbar_wait(all_done, 0, nullptr));
  }
  fence_before();
  __syncthreads();
  if (warp == kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// The heads of a Q tile: of the divisors of G, the one whose tiles of
// floor(128 / heads) tokens waste the fewest rows on sequences of the mean
// length; the most heads where several do (fewer K and V loads a row).
int heads_of_tile(int64_t G, int64_t B, int64_t Tq) {
  const double mean = B > 0 ? (double)Tq / (double)B : 1.0;
  int best = 1;
  double most = -1.0;
  for (int hg = 1; hg <= G && hg <= kRows; ++hg) {
    if (G % hg) continue;
    const double tpt = kRows / hg, tiles = mean <= tpt ? 1.0 : mean / tpt;
    const double use = mean * hg / (kRows * (tiles < 2.0 ? (double)(int)(tiles + 0.999) : tiles + 0.5));
    if (use >= most) most = use, best = hg;
  }
  return best;
}

template <int D>
cudaError_t launch(const PrefillArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  Args p;
  p.a = a;
  p.G = (int)(a.Hq / a.Hkv);
  p.hg = heads_of_tile(p.G, a.B, a.Tq);
  p.tpt = kRows / p.hg;
  CUtensorMap mq, mk, mv;
  cudaError_t e = encode_tma_heads(&mq, a.q, D, a.Hq, a.Tq, a.q_stride, p.hg, p.tpt);
  if (a.Tk > 0) {
    if (e == cudaSuccess) e = encode_tma_heads(&mk, a.k, D, a.Hkv, a.Tk, a.k_stride, 1, kKeys);
    if (e == cudaSuccess) e = encode_tma_heads(&mv, a.v, D, a.Hkv, a.Tk, a.v_stride, 1, kKeys);
  } else {
    mk = mv = mq;  // never loaded from
  }
  if (e != cudaSuccess) return e;
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidDevice;
  auto kern = attn_prefill_kernel<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // every sequence has at most one run that is not whole
  const int64_t run = C::kTiles * p.tpt, items = a.Tq / run + (a.B < a.Tq ? a.B : a.Tq);
  const int64_t heads = a.Hkv * (p.G / p.hg);
  if (items > INT32_MAX || heads > 65535) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)items, (unsigned)heads), dim3(C::kThreads), C::kSmem, st, mq,
                    mk, mv, p, status);
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
