// attn_tc.cuh -- what the attention kernels on the 5th-generation tensor cores
// share: bounded waits, descriptors, MMAs and TMEM accesses (inline PTX), packed
// fp32 arithmetic, and the shape of a Q tile.
#pragma once

#include <cuda_bf16.h>

#include "async_util.cuh"
#include "packed.cuh"
#include "ptq_internal.cuh"

namespace ptq {

constexpr int kRows = 128;  // rows of a Q tile
constexpr int kKeys = 128;  // keys of a K and V tile
constexpr float kSlack = 8.0f;  // log2 of the largest P
constexpr int64_t kSms = 152;

__device__ __forceinline__ int clamped(int v, int hi) { return min(max(v, 0), hi); }

// What the warps of a CTA tell one another beside the barriers, in one word: kAborted,
// a wait ran out; kBusy for each warp at something that may take long.
constexpr int kAborted = 1, kBusy = 2;

// A bounded wait, in few instructions: the warps' roles together are larger than
// the instruction cache.  It gives up after kWaitLimit polls (of 1.5 us) while no
// warp is busy.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* state) {
  const uint32_t at = smem_addr(bar);
#pragma unroll 1
  for (uint32_t i = kWaitLimit; i > 0; --i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (done) return true;
    const int now = *state;
    if (__builtin_expect(now != 0, 0)) {
      if (now & kAborted) return false;
      i = kWaitLimit;
    }
  }
  return false;
}

// A warp's stretch of being busy.
struct Busy {
  int* state;
  __device__ __forceinline__ explicit Busy(volatile int* at) : state(const_cast<int*>(at)) {
    if ((threadIdx.x & 31) == 0) atomicAdd(state, kBusy);
  }
  __device__ __forceinline__ ~Busy() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) atomicSub(state, kBusy);
  }
};

// N (2, 4 or 8) consecutive values, aligned to their size.
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&x)[N]) {
  uint32_t w[N / 2];
  if constexpr (N == 2) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (N == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    x[i] = __uint_as_float(w[i / 2] << 16);
    x[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
  }
}

// ---- tensor core -------------------------------------------------------------------

// Shared-memory descriptor of a 128-byte-swizzled tile: 8-row atoms 1024
// bytes apart; lead: bytes between column blocks of 64 (N-major operands).  The
// upper word is the same for all, the lower moves along by 16 bytes a unit.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr, uint32_t lead) {
  return (addr >> 4) | (lead >> 4) << 16;
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
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, %4;\n}" ::"r"(d), "r"(a), "r"(b),
      "r"(id), "n"(kAdd ? 1 : 0), "n"(kDescHi)
      : "memory");
}
template <bool kAdd>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n .reg .b64 db;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, %4;\n}" ::"r"(d), "r"(a), "r"(b),
      "r"(id), "n"(kAdd ? 1 : 0), "n"(kDescHi)
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : PTQ_R8(v, 0), PTQ_R8(v, 8)
      : "r"(addr));
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
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 bytes of a row, whose alignment is 16 or 32.
__device__ __forceinline__ void store32(char* p, const uint32_t* w, bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), PTQ_W8(w, 0)
                 : "memory");
  } else {
    uint4* q = reinterpret_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The heads of a Q tile: of the divisors of G, the one whose tiles of
// floor(128 / heads) tokens waste the fewest rows on sequences of the mean
// length (one sequence: on it; several: half a run each); the most heads where
// several do (fewer K and V loads a row).  Against one head a tile, five of
// 128: 16 prompts of 25 tokens 6.4 us for 15.4, of 550 68 for 91; one of 8192
// takes 450 either way.
inline int heads_of_tile(int64_t G, int64_t B, int64_t Tq, int tiles) {
  const double mean = (double)Tq / (double)(B < 1 ? 1 : B < Tq ? B : Tq);
  int best = 1;
  double most = -1.0;
  for (int hg = 1; hg <= G && hg <= kRows; ++hg) {
    if (G % hg) continue;
    const int64_t tpt = kRows / hg, run = tiles * tpt;
    const double rows = B == 1 ? (double)((Tq + tpt - 1) / tpt * tpt)
                        : mean < (double)run ? (mean > (double)tpt ? (double)run : (double)tpt)
                                             : mean + 0.5 * (double)run;
    const double use = mean / rows * (double)(hg * tpt) / kRows;
    if (use >= most) most = use, best = hg;
  }
  return best;
}

}  // namespace ptq
