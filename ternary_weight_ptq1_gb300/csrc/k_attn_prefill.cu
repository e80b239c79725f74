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
// buffers.  Either way the tensor core has one S's products in work while the
// softmax of the other runs.  A slot of TMEM holds S, then P, and one thread
// issues all of a slot's MMAs, which run in order: that alone keeps P from
// being overwritten before it is read.
//
// Warps: four for the softmax of each Q tile (a thread holds a row: its
// maximum and sum need no shuffle), one that issues the TMA loads, one for
// each Q tile that issues its MMAs.  The maximum that P refers to moves only when a row's
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
  // A K or V tile passes through the ring in one unit, or two: K by columns,
  // V by keys, as the products use them up.
  static constexpr int kUnits = D == 256 ? 2 : 1;
  static constexpr int kCols = D / kUnits;           // columns of a K unit
  static constexpr int kVKeys = kKeys / kUnits;      // keys of a V unit
  static constexpr int kUnit = kKeys * kCols * 2;    // bytes
  static constexpr int kRing = D == 64 ? 8 : 5;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSoftmax = 4 * kTiles;        // softmax warps
  static constexpr int kThreads = 32 * (kSoftmax + 4);  // whole groups of four warps
  // Registers a thread: 384 threads get 168 each at launch (64,512 in all);
  // 256 softmax threads take 208 and 128 others keep 80 (63,488).
  static constexpr bool kSplitRegs = kTiles == 2;
  static constexpr int kOffRing = kTiles * kQ;
  static constexpr int kOffBar = kOffRing + kRing * kUnit;
  // P over S's columns; at head_dim 64 TMEM has room for P beside S, and the
  // next S is in work as soon as this one has been read.
  static constexpr bool kApart = D == 64;
  // full[kRing] empty[kRing] q s[2] read[2] p[2][2] o[2] pv[2] turn[2] done
  static constexpr int kBars = 2 * kRing + 1 + 2 + 2 + 4 + 2 + 2 + 2 + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 64;
};
static_assert(Cfg<128>::kSmem <= 227 * 1024 && Cfg<256>::kSmem <= 227 * 1024, "shared memory");
// A unit is as many bytes as its boxes of 64 columns bring.
static_assert(Cfg<256>::kUnit == kKeys * Cfg<256>::kCols * 2 &&
                  Cfg<256>::kUnit == Cfg<256>::kVKeys * 256 * 2 &&
                  Cfg<64>::kUnit == Cfg<64>::kVKeys * 64 * 2, "ring units");

struct Args {
  PrefillArgs a;
  int G, hg, tpt;  // query heads of a kv head; heads and tokens of a Q tile
  int heads;       // head blocks in all
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

// kAdd: onto what the accumulator holds.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, %4;" ::"r"(d), "l"(a), "l"(b),
               "r"(id), "n"(kAdd ? 1 : 0)
               : "memory");
}
template <bool kAdd>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id) {
  asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, %4;" ::"r"(d), "r"(a), "l"(b),
               "r"(id), "n"(kAdd ? 1 : 0)
               : "memory");
}
// One lane of the converged warp, the same each time.
__device__ __forceinline__ bool elected() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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
  // of a slot: S written, S read (kApart), the first and second half of P
  // written; of a Q tile: O final, a product with V done (not where S's
  // arrival says it), its turn to issue
  uint64_t *s_full = q_full + 1, *s_read = s_full + 2, *p_full = s_read + 2, *o_full = p_full + 4,
           *pv_done = o_full + 2, *turn = pv_done + 2, *all_done = turn + 2;
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
        mbar_init(empty + i, kTiles);
      }
      mbar_init(q_full, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(s_full + i, 1);
        mbar_init(s_read + i, 4);  // the four softmax warps of a tile
        mbar_init(p_full + 2 * i, 4);
        mbar_init(p_full + 2 * i + 1, 4);
        mbar_init(o_full + i, 1);
        mbar_init(pv_done + i, 1);
        mbar_init(turn + i, 1);
      }
      mbar_init(all_done, kTiles);
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  } else if (warp == 0) {
    pdl_wait();
    int b = -1, t = 0;
    if (!find_item(a, kTiles * p.tpt, blockIdx.x / p.heads, &b, &t)) b = -1;
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
    // heads fastest: the long items of all of them come first
    const int blocks = p.G / p.hg, head = (int)blockIdx.x % p.heads;
    const int h = head / blocks, hq0 = h * p.G + (head % blocks) * p.hg;
    // Q tile s: queries tok(s) .. tok(s) + tpt - 1 of the sequence; keys of its
    // last query; K tiles
    int first[kTiles], keys[kTiles], n[kTiles];
#pragma unroll
    for (int s = 0; s < kTiles; ++s) {
      first[s] = (item[1] * kTiles + s) * p.tpt;
      const int last = min(first[s] + p.tpt, sp.nq) - 1;
      keys[s] = a.causal ? min(sp.nk, sp.nk - sp.nq + last + 1) : sp.nk;
      n[s] = first[s] < sp.nq && keys[s] > 0 ? (keys[s] + kKeys - 1) / kKeys : 0;
    }
    int most = n[0];
    if (kTiles == 2) most = max(most, n[kTiles - 1]);
    const uint32_t ring = smem_addr(smem + C::kOffRing), qs = smem_addr(smem);
    bool ok = true;

    if (warp >= C::kSoftmax) {
      if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }
    if (warp == kLoad) {
      // ---- loads: Q, then K and V tiles through the ring in the order of their use:
      // K_0 V_0 K_1 V_1 ..., or with one Q tile K_0 K_1 V_0 K_2 V_1 ... --------------
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
        auto load = [&](const CUtensorMap* map, int x, int y, int rows, int blocks) {
          const int st = u % C::kRing, round = u / C::kRing;
          if (round > 0) ok = mbar_wait(empty + st, (round - 1) & 1, abort_flag);
          if (!ok) return;
          mbar_expect_tx(full + st, C::kUnit);
          for (int c = 0; c < blocks; ++c)  // boxes of 64 columns
            tma_3d(ring + st * C::kUnit + c * rows * 128, map, x + 64 * c, h, y, full + st);
          ++u;
        };
        auto load_k = [&](int j) {
          for (int k = 0; k < C::kUnits && ok; ++k)
            load(&map_k, k * C::kCols, sp.k0 + j * kKeys, kKeys, C::kCols / 64);
        };
        auto load_v = [&](int j) {
          for (int k = 0; k < C::kUnits && ok; ++k)
            load(&map_v, 0, sp.k0 + j * kKeys + k * C::kVKeys, C::kVKeys, D / 64);
        };
        load_k(0);
        for (int j = 0; j < most && ok; ++j) {
          if (kTiles == 1 && j + 1 < most) load_k(j + 1);
          load_v(j);
          if (kTiles == 2 && j + 1 < most) load_k(j + 1);
        }
        // whatever becomes of the MMAs, the copies land before the CTA ends
        for (int v = max(0, u - C::kRing); v < u; ++v)
          static_cast<void>(mbar_wait(full + v % C::kRing, (v / C::kRing) & 1, nullptr));
        static_cast<void>(mbar_wait(q_full, 0, nullptr));
      }
    } else if (warp >= kMma && warp < kMma + kTiles) {
      // ---- MMAs.  The warp stays converged and one lane issues each product in
      // straight-line code.  The tensor core takes few MMAs ahead, so a pause in
      // the issue is a pause in the products: with two Q tiles each has an issuing
      // warp of its own, and one waits for barriers while the other's MMAs run ----
      const int s = warp - kMma, tiles = n[s];
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && __all_sync(~0u, mbar_wait(bar, phase & 1, abort_flag));
      };
      auto arrived = [&](int u) { wait(full + u % C::kRing, u / C::kRing); };  // ring unit u
      // first unit of K_j and V_j (with one Q tile, past the last K there is no
      // K_(j + 1) before V_j)
      auto k_unit = [&](int j) { return (kTiles == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1) * C::kUnits; };
      auto v_unit = [&](int j) {
        return (kTiles == 2 || j == most - 1 ? 2 * j + 1 : 2 * j + 2) * C::kUnits;
      };
      // A K or V tile that the other Q tile does not use is released for both.
      auto release = [&](int j, int st) {
        mma_commit(empty + st);
        if (kTiles == 2 && j >= n[kTiles - 1 - s]) mma_commit(empty + st);
      };
      // S of tile j into its slot: unit k of the columns
      auto qk = [&](int j, int k) {
        const int slot = kTiles == 1 ? j & 1 : s, st = (k_unit(j) + k) % C::kRing;
        const uint64_t qd = tile_desc(qs + s * C::kQ + k * (C::kCols / 64) * kRows * 128, 16);
        const uint64_t kd = tile_desc(ring + st * C::kUnit, 16);
#pragma unroll
        for (int c = 0; c < C::kCols / 64; ++c)  // descriptors count 16 bytes
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = c * (kRows * 128 / 16) + 2 * e;
            if (k == 0 && c == 0 && e == 0)
              mma_ss<false>(tmem + slot * kKeys, qd + at, kd + at, idesc<kKeys, false>());
            else
              mma_ss<true>(tmem + slot * kKeys, qd + at, kd + at, idesc<kKeys, false>());
          }
        release(j, st);
        if (k == C::kUnits - 1) mma_commit(s_full + slot);
      };
      // O += P V of tile j over its first or second 64 keys
      auto pv = [&](int j, int half) {
        const int slot = kTiles == 1 ? j & 1 : s;
        const uint32_t pa = tmem + (C::kApart ? 384 + slot * 64 : slot * kKeys) + 32 * half;
        const uint32_t d = tmem + 2 * kKeys + s * D;
        const int st = (v_unit(j) + (C::kUnits == 2 ? half : 0)) % C::kRing;
        const uint64_t vd = tile_desc(ring + st * C::kUnit + (C::kUnits == 2 ? 0 : 8192 * half),
                                      C::kVKeys * 128);
        if (j > 0 || half > 0)
          mma_ts<true>(d, pa, vd, idesc<D, true>());
        else
          mma_ts<false>(d, pa, vd, idesc<D, true>());
#pragma unroll
        for (int e = 1; e < 4; ++e)  // 16 keys: 8 columns of P, 2048 bytes of V
          mma_ts<true>(d, pa + 8 * e, vd + 128 * e, idesc<D, true>());
        if (half == 1 || C::kUnits == 2) release(j, st);
        if (half == 1) {
          if (kTiles == 1 || C::kApart) mma_commit(pv_done + s);
          if (j == tiles - 1) mma_commit(o_full + s);
        }
      };
      if (tiles > 0) {
        wait(q_full, 0);
        auto scores = [&](int j) {
#pragma unroll
          for (int k = 0; k < C::kUnits; ++k) {
            arrived(k_unit(j) + k);
            fence_after();
            if (ok && elected()) qk(j, k);
            __syncwarp();
          }
        };
        scores(0);
        for (int j = 0; j < tiles && ok; ++j) {
          const bool more = j + 1 < tiles;
          const int slot = kTiles == 1 ? j & 1 : s, use = kTiles == 1 ? j >> 1 : j;
          if (more && kTiles == 1) scores(j + 1);
          if (more && C::kApart) {
            wait(s_read + slot, use);
            scores(j + 1);
          }
          for (int k = 0; k < C::kUnits; ++k) arrived(v_unit(j) + k);
          constexpr bool kAfter = kTiles == 2 && !C::kApart;  // the next S goes where P was
          if (more && kAfter) arrived(k_unit(j + 1));
          wait(p_full + 2 * slot, use);
          // Two Q tiles take turns: issued side by side their MMAs would alternate,
          // both S would arrive together and the tensor core would stand still
          // during both softmaxes (540 for 442 us, 8192 tokens).
          if (kAfter) {
            if (s == 1 && j < n[0]) wait(turn + s, j);
            if (s == 0 && j > 0 && j - 1 < n[kTiles - 1]) wait(turn + s, j - 1);
          }
          fence_after();
          if (ok && elected()) pv(j, 0);
          __syncwarp();
          wait(p_full + 2 * slot + 1, use);
          fence_after();
          if (ok && elected()) {
            pv(j, 1);
            if (kAfter) {
              if (more) qk(j + 1, 0);
              mbar_arrive(turn + 1 - s);
            }
          }
          __syncwarp();
        }
      }
      if (elected()) mma_commit(all_done);
      __syncwarp();
    } else if (warp < C::kSoftmax) {
      // ---- softmax: thread = row of Q tile s ----------------------------------------
      if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
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
      bool ready = false;
      uint64_t sum2[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
      for (int j = 0; j < n[s] && ok; ++j) {
        const int slot = kTiles == 1 ? j & 1 : s, use = kTiles == 1 ? j >> 1 : j;
        const uint32_t at = tmem + lanes + slot * kKeys;
        const uint32_t p_at = C::kApart ? tmem + lanes + 384 + slot * 64 : at;
        ok = __all_sync(~0u, ready || mbar_wait(s_full + slot, use & 1, abort_flag));
        if (!ok) break;
        fence_after();
        uint32_t v[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(at + c, v + c);
        tmem_wait_ld();
        if constexpr (C::kApart) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_read + slot);
        }
        if ((j + 1) * kKeys > all_see) {
          const int left = sees - j * kKeys;
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c >= left) v[c] = 0xff800000u;
        }
        float top[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top[e] = max3(__uint_as_float(v[3 * e]), __uint_as_float(v[3 * e + 1]),
                        __uint_as_float(v[3 * e + 2]));
#pragma unroll
        for (int c = 12; c < kKeys; c += 2)  // 116 more in pairs, 14 or 15 a chain
          top[c / 2 % 4] = max3(top[c / 2 % 4], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
        const float t2 = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale2;
        if (j == 0) {
          m = t2;
        } else if (__any_sync(~0u, t2 > m + kSlack)) {
          // O moves to the new maximum once the product with the tile before is
          // done (where S follows P, S says so)
          if constexpr (kTiles == 1 || C::kApart) {
            ok = __all_sync(~0u, mbar_wait(pv_done + s, (j - 1) & 1, abort_flag));
            if (!ok) break;
          }
          const float mn = t2 > m + kSlack ? t2 : m;
          const float f = m == kNegInf ? 0.0f : exp2_fast(m - mn);
          m = mn;
          fence_after();
          float lo, hi;
          unpair(sum2[0], lo, hi);
          sum2[0] = pair(lo * f, hi * f);
          unpair(sum2[1], lo, hi);
          sum2[1] = pair(lo * f, hi * f);
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
        auto half_p = [&](int c) {  // keys c .. c + 63
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            unpair(fma2(pair(__uint_as_float(v[c + 2 * e]), __uint_as_float(v[c + 2 * e + 1])), ss, zz), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum2[e & 1] = add2(sum2[e & 1], pair(x0, x1));
            w[e] = bf16x2(x0, x1);
          }
          if constexpr (C::kApart)  // the product with the tile before has read its P
            if (c == 0 && j > 0)
              ok = __all_sync(~0u, mbar_wait(pv_done + s, (j - 1) & 1, abort_flag));
          tmem_st32(p_at + c / 2, w);
        };
        auto publish = [&](int half) {
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 2 * slot + half);
        };
        // The product with V starts on the first half.  The branch is worth more
        // than the work it saves in a last tile: without it the compiler computes
        // both halves before it stores the first.
        half_p(0);
        publish(0);
        {  // whether the next S has arrived: asked now, used at the top
          const int nj = j + 1, nslot = kTiles == 1 ? nj & 1 : s, nuse = kTiles == 1 ? nj >> 1 : nj;
          ready = nj < n[s] && mbar_test(s_full + nslot, nuse & 1);
        }
        if (keys[s] - j * kKeys > 64) {
          half_p(64);
        } else {
          const uint32_t none[32] = {};
          tmem_st32(p_at + 32, none);
        }
        publish(1);
      }

      // ---- epilogue ----------------------------------------------------------------
      float lo, hi;
      unpair(add2(sum2[0], sum2[1]), lo, hi);
      const float l = lo + hi;
      const int64_t tq = sp.q0 + tok;
      const int hq = hq0 + row % p.hg;
      const bool some = n[s] > 0;
      if (ok && some) ok = __all_sync(~0u, mbar_wait(o_full + s, 0, abort_flag));
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
          if (some) {
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
    if (e == cudaSuccess) e = encode_tma_heads(&mv, a.v, D, a.Hkv, a.Tk, a.v_stride, 1, C::kVKeys);
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
  if (items * heads > INT32_MAX) return cudaErrorInvalidValue;
  p.heads = (int)heads;
  return launch_pdl(kern, dim3((unsigned)(items * heads)), dim3(C::kThreads), C::kSmem, st, mq,
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
