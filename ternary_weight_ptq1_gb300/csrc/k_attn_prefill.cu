// k_attn_prefill.cu -- attention of packed prompts on the 5th-generation
// tensor cores.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - m),  O = P V,  out = O / sum P
//
// 4 head_dim operations a visible (query, key) pair and query head against
// one exponential.  On long prompts the tensor cores and the shared memory that
// feeds them bound it (at head_dim 64 the exponentials): a step of 128 keys and
// two Q tiles of 128 columns is 2048 clocks of products, which read 192 KB and
// for which 64 KB arrive, 2000 clocks at 128 bytes each; a step of one Q tile
// of 256 columns is 2048 clocks of products and 320 KB, 2500 clocks.  On short
// ones the chain S, softmax, P, O of each item's few steps bounds it.
//
// Measured in CUDA graphs, causal, bf16: 8192 tokens of 8 x 5 heads of 128 in 453 us
// (1520 TFLOP/s, 82% of a library product's rate) over some ms, 473 over longer runs; of
// 4 x 6 heads of 256 in 546 (1510), of 4 x 7 of 64 in 261 (920); 16 prompts of up to
// 1100 tokens in 76 us (790); two of 460 and 479 over prefixes, 3518 and 2667 keys,
// 4 x 6 of 256, in 77 us (850, on 1.2 items an SM); 77 tokens in 7.5 us.
//
// Tile.  128 rows of Q are tpt tokens of hg query heads that share a kv head
// (row = token * hg + head, one TMA box), against tiles of 128 keys.  S and O
// live in TMEM; P goes back there as bf16 over S's columns and is the A
// operand of the second product, so only K and V pass through shared memory.  (A and
// B have one type, and V is bf16: P keeps 8 bits.  A second bf16 term of it would add
// half to the products.  Its sum is taken in fp32, before the rounding.)
// A CTA holds two Q tiles (head_dim up to 128), neighbours in the sequence,
// that share each K and V tile; at head_dim 256 one Q tile whose S has two
// buffers.  Either way the tensor core has one S's products in work while the
// softmax of the other runs.  A slot of TMEM holds S, then P, and one thread
// issues all of a slot's MMAs, which run in order: that alone keeps P from
// being overwritten before it is read.
//
// Warps: four for the softmax of each Q tile (a thread holds a row: its
// maximum and sum need no shuffle), four that store the output while the next
// item is in work, one that issues the TMA loads, one for each Q tile that
// issues its MMAs, one that finds the CTA's next item.  The maximum that P
// refers to moves only when a row's grows by more than 2^8 over it: P up to 2^8
// costs fp32 sums nothing, and rescaling O (TMEM to registers and back) becomes
// rare.
//
// One CTA an SM goes through items (two neighbouring Q tiles, or one, of one
// sequence and head block), the longest first, dealt out there and back.  Where
// the items are few and the keys long, the keys are cut into parts whose sums
// a second kernel joins in order.
//
// A key that a row does not see has P = 0, and 0 times a non-finite value is NaN.
// The values past a long sequence's end are cleared in shared memory; rows that a
// value hidden from them has spoilt are computed again over the keys they see (8192
// tokens, 8 x 5 heads of 128, 0.46 ms: with the last token's value infinite 18 ms,
// with the first one's, which every row sees, 0.64).
//
// All roles' code together is larger than the instruction cache: what runs once
// an item is kept short, in loops where that costs nothing (a fifth of the
// fetches missed when 74 KB were in use; of the 52 KB besides what spoilt rows and
// ends of sequences take, 4% do, and the packed prompts went from 101 us to 76).
// Only the products and the softmax of a tile are unrolled: the MMAs of both halves
// of P issued by one loop, whose operands are then no constants, took 583 us for 466
// at 8192 tokens.
//
// Every wait is bounded, to some 6 s in which no warp computes rows again; one that
// runs out raises the device status word and the CTA drains what it has in flight and
// exits.
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
  static constexpr int kThreads = 32 * (kSoftmax + 8);  // four to store, four others
  // Registers a thread.  Two Q tiles: 512 threads get 128 each at launch (65,536
  // in all); 256 softmax threads take 168, 128 that store keep 96 and 128 others
  // 80 (65,536).  One: 384 get 168 (64,512); 128 take 232, 128 keep 128, 128 keep
  // 104 (59,392).
  static constexpr int kRegsSoftmax = kTiles == 2 ? 168 : 232;
  static constexpr int kRegsStore = kTiles == 2 ? 96 : 128;
  static constexpr int kRegsOther = kTiles == 2 ? 80 : 104;
  static constexpr int kOffRing = kTiles * kQ;
  static constexpr int kOffBar = kOffRing + kRing * kUnit;
  // full[kRing] empty[kRing] q[2] q free[2] s[2] p[2][2] o[2] o free[2] pv[2] turn[2]
  // item full[2] item empty[2] sums full[2] sums empty[2] tail full done
  static constexpr int kBars = 2 * kRing + 4 + 2 + 4 + 2 + 2 + 2 + 2 + 2 + 2 + 2 + 2 + 1 + 1;
  static constexpr int kOffItem = (kOffBar + 8 * kBars + 15) / 16 * 16;
  static constexpr int kOffSums = kOffItem + 2 * 64;  // (maximum, sum) of each row
  static constexpr int kOffMisc = kOffSums + kTiles * kRows * 8;
  static constexpr int kSmem = kOffMisc + 16;
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
  Divider by_per, by_heads, by_G, by_hg;  // by_per: head blocks times parts
  Divider by_run;  // queries of an item: the Q tiles' tokens
  int ways;        // through the sequences, that the planning warp may go
  int splits;      // parts the keys of each item are cut into
  float* part;     // splits > 1: [splits][Tq Hq][D] output sums, and the (maximum,
  float2* ml;      // sum) they refer to, [splits][Tq Hq]
};

// A CTA's next piece of work: Q tiles of one sequence and head block, over one
// part of the keys.  b < 0: no more.
struct Item {
  int b, q0, nq, k0, nk;  // the sequence's place
  int first;              // first query of Q tile 0
  int h, hq0;             // kv head, first query head
  int split;
  int lo;                 // the part's first tile of 128 keys
  int n[2];               // its tiles that Q tile s sees some key of
  int keys[2];            // keys the last query of Q tile s sees
};
static_assert(sizeof(Item) <= 64, "its place in shared memory");

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

struct Span {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Span span_of(const PrefillArgs& a, int b) {
  const int Tq = (int)a.Tq, Tk = (int)a.Tk;
  const int q0 = clamped(__ldg(a.cu_q + b), Tq), q1 = clamped(__ldg(a.cu_q + b + 1), Tq);
  const int k0 = clamped(__ldg(a.cu_k + b), Tk), k1 = clamped(__ldg(a.cu_k + b + 1), Tk);
  return {q0, max(0, q1 - q0), k0, max(0, k1 - k0)};
}

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

// Query rows by a warp, kGroup rows and 32 keys at a time (a lane's own key for the
// scores, a lane's own columns for the outputs): those of the lanes `todo` (a lane a
// row: query t, head hq, over keys [k0, end)).  (Groups of two need 64 registers, 100 at
// head_dim 256, groups of four more than kRegsStore, which the function has to fit.)
constexpr int kGroup = 2;
template <int D>
__device__ __forceinline__ void attend_rows(const Args& p, int split, unsigned todo, int t, int hq, int h,
                                            int k0, int end) {
  constexpr int N = D / 32, kBatch = D == 256 ? 4 : 8;
  const PrefillArgs& a = p.a;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  while (todo) {
    RowState<D> r[kGroup];
    const uint16_t* q[kGroup];
    int64_t row[kGroup];
    int ends[kGroup], most = k0;
    int who = 0;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {  // the last row again where there are no more
      if (todo) who = __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t tg = __shfl_sync(~0u, t, who);
      const int hg = __shfl_sync(~0u, hq, who);
      q[g] = a.q + tg * a.q_stride + (int64_t)hg * D;
      row[g] = tg * a.Hq + hg;
      ends[g] = __shfl_sync(~0u, end, who);
      most = max(most, ends[g]);
    }
#pragma unroll 1
    for (int j0 = k0; j0 < most; j0 += 32) {
      float s[kGroup] = {}, w[kGroup];
      const uint16_t* key = a.k + (int64_t)min(j0 + lane, most - 1) * a.k_stride + (int64_t)h * D;
#pragma unroll 4
      for (int d = 0; d < D; d += 8) {
        float x[8];
        load_bf16(key + d, x);
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
          float y[8];
          load_bf16(q[g] + d, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[g] = fmaf(x[i], y[i], s[g]);
        }
      }
#pragma unroll
      for (int g = 0; g < kGroup; ++g)
        w[g] = r[g].weigh(j0 + lane < ends[g] ? s[g] * (a.scale * kLog2e) : kNegInf);
      const uint16_t* value = a.v + (int64_t)j0 * a.v_stride + (int64_t)h * D + lane * N;
#pragma unroll 1
      for (int j = 0; j < min(32, most - j0); j += kBatch) {
        float v[kBatch][N];  // loaded together
#pragma unroll
        for (int e = 0; e < kBatch; ++e) load_bf16(value + (int64_t)min(j + e, most - 1 - j0) * a.v_stride, v[e]);
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            const float wj = __shfl_sync(~0u, w[g], j + e);
            if (j0 + j + e < ends[g]) {  // (0 times a hidden value may be NaN)
#pragma unroll
              for (int i = 0; i < N; ++i) r[g].o[i] = fmaf(wj, v[e][i], r[g].o[i]);
            }
          }
      }
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      float l = r[g].l;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(~0u, l, i);
      if (p.splits > 1) {
        const int64_t at = (int64_t)split * a.Tq * a.Hq + row[g];
        if (lane == 0) p.ml[at] = make_float2(r[g].m, l);
#pragma unroll
        for (int i = 0; i < N; ++i) p.part[at * D + lane * N + i] = r[g].o[i];
        continue;
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int i = 0; i < N; ++i)
        a.out[row[g] * D + lane * N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(r[g].o[i] * inv));
    }
  }
}

// The rows `again` of a warp (a lane a row: query t, head hq, which sees `sees` of
// the part's `end` keys from key0 on) whose output is not finite though their sum
// is.  A value that a row sees and that is not finite leaves its column so, rightly.
// The row is computed again where a column has none of those, but one among the
// hidden keys of the tiles (0 times it is NaN), and where no value explains it
// (P may be 2^8 times a probability, and the sums of large values overflow).
template <int D>
__device__ __noinline__ void repair(const Args& p, int split, unsigned again, int t, int hq, int sees, int h,
                                    int key0, int end, volatile int* state) {
  constexpr int N = D / 32;
  const Busy busy(state);
  const PrefillArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const bool mine = again >> lane & 1;
  const int least = __reduce_min_sync(~0u, mine ? sees : end), most = __reduce_max_sync(~0u, mine ? sees : 0);
  const uint16_t* value = a.v + (int64_t)key0 * a.v_stride + (int64_t)h * D + lane * N;
  // of this lane's columns: the last hidden key and the first seen one that are not finite
  int last[N], first[N];
#pragma unroll
  for (int i = 0; i < N; ++i) last[i] = -1, first[i] = end;
#pragma unroll 4
  for (int j = least; j < end; ++j) {
    float v[N];
    load_bf16(value + (int64_t)j * a.v_stride, v);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(fabsf(v[i]) < -kNegInf)) last[i] = j;
  }
#pragma unroll 1
  for (int j0 = 0; j0 < most; j0 += 16) {
#pragma unroll 4
    for (int j = j0; j < min(j0 + 16, most); ++j) {
      float v[N];
      load_bf16(value + (int64_t)j * a.v_stride, v);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(fabsf(v[i]) < -kNegInf)) first[i] = min(first[i], j);
    }
    bool some = false, open = false;  // found one; a column that a hidden key spoils has none yet
#pragma unroll
    for (int i = 0; i < N; ++i) {
      some |= first[i] < end;
      open |= first[i] == end && last[i] >= 0;
    }
    if (__any_sync(~0u, some) && !__any_sync(~0u, open)) break;
  }
  unsigned todo = 0;
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int who = __ffs(again) - 1, n = __shfl_sync(~0u, sees, who);
    bool known = false, spoiled = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      known |= first[i] < n;
      spoiled |= first[i] >= n && last[i] >= n;
    }
    if (__any_sync(~0u, spoiled) || !__any_sync(~0u, known)) todo |= 1u << who;
  }
  attend_rows<D>(p, split, todo, t, hq, h, key0, key0 + sees);
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// A ring unit of values with a sequence's end in it, for the tensor core to see zeros
// past the `left` keys (64 or 128 from y on) that are the sequence's: it arrives at
// `bar`, is cleared there and handed over at `full`.  False: the wait ran out.
//
// Sequences of more than kClear keys alone are given that: without it their rows (under
// a causal mask the last ones, else all) are computed again when the next sequence's
// values are not finite.  For short ones that is little, and the wait takes each item
// 0.5 us (40 prompts of up to 300 tokens, 4 x 7 of 64, all keys: 29.6 us for 28.1).
constexpr int kClear = 1024;
template <int D>
__device__ __noinline__ bool load_tail(const CUtensorMap* map, uint32_t unit, uint64_t* bar, uint32_t parity,
                                       uint64_t* full, int h, int y, int left, volatile int* state) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  if (left > 0) {
    if (lane == 0) {
      mbar_expect_tx(bar, C::kUnit);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) tma_3d(unit + c * C::kVKeys * 128, map, 64 * c, h, y, bar);
    }
    if (!__all_sync(~0u, bar_wait(bar, parity, state))) {
      static_cast<void>(mbar_wait(bar, parity, nullptr));  // the copy lands
      return false;
    }
  }
#pragma unroll 1
  for (uint32_t i = max(0, left) * 128 + lane * 16; i < C::kVKeys * 128; i += 512)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(unit + c * C::kVKeys * 128 + i), "r"(0)
                   : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}

// ---- the order of the work -----------------------------------------------------------
// Sequences are cut into runs of `run` queries.  The runs that come late in
// their sequence (under a causal mask those with the most keys) are first: band
// by band of levels downwards, through the sequences in each band, and downwards
// in each sequence's part of the band.  One warp walks them, each time further on,
// 32 sequences a step; a band is one level, or as many as keep the walk to kSteps
// steps (or to one way through the sequences).
constexpr int kSteps = 4096;

struct Walk {
  int base;      // the band's first level
  int band;      // its levels
  int b0;        // the next 32 sequences
  int before;    // runs before them
  int all;       // runs in all
  int first;     // of this lane's sequence among the first 32
};

// The runs of sequence b.
__device__ __forceinline__ int runs_of(const Args& p, int b) {
  const PrefillArgs& a = p.a;
  if (b >= (int)a.B) return 0;
  const int Tq = (int)a.Tq;
  const int n = max(0, clamped(__ldg(a.cu_q + b + 1), Tq) - clamped(__ldg(a.cu_q + b), Tq));
  return p.by_run(n + p.by_run.d - 1);
}

__device__ __forceinline__ Walk walk_from_top(const Args& p) {
  const int lane = threadIdx.x & 31, first = runs_of(p, lane);
  int most = first, all = first;
#pragma unroll 1
  for (int b = 32 + lane; b < (int)p.a.B; b += 32) {
    const int n = runs_of(p, b);
    most = max(most, n);
    all += n;
  }
  most = (int)__reduce_max_sync(~0u, most);
  all = (int)__reduce_add_sync(~0u, all);
  // most / band ways through the sequences (no division where a band is a level)
  if (most <= p.ways) return {most - 1, 1, 0, 0, all, first};
  const int band = (most + p.ways - 1) / p.ways;
  return {(most - 1) / band * band, band, 0, 0, all, first};
}

// The sequence and level of run i in that order; false: there are not so many.
// i grows from call to call.
__device__ __forceinline__ bool walk_to(const Args& p, int i, Walk& w, int* seq, int* level) {
  const int lane = threadIdx.x & 31;
  if (i >= w.all) return false;
#pragma unroll 1
  for (; w.base >= 0; w.base -= w.band, w.b0 = 0) {
#pragma unroll 1
    for (; w.b0 < (int)p.a.B; w.b0 += 32) {
      const int mine = min(max((w.b0 ? runs_of(p, w.b0 + lane) : w.first) - w.base, 0), w.band);
      int end = mine;  // the sum up to this lane
      if (w.band == 1) {
        end = __popc(__ballot_sync(~0u, mine) & (~0u >> (31 - lane)));
      } else {
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, end, d);
          if (lane >= d) end += o;
        }
      }
      const int in = i - w.before;
      const unsigned at = __ballot_sync(~0u, in < end);
      if (at) {
        const int who = __ffs(at) - 1;
        *seq = w.b0 + who;
        *level = w.base + __shfl_sync(~0u, end, who) - 1 - in;
        return true;
      }
      w.before += __shfl_sync(~0u, end, 31);
    }
  }
  return false;
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

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args p,
                        int* status) {
  using C = Cfg<D>;
  constexpr int kTiles = C::kTiles;
  constexpr bool kAfter = kTiles == 2;  // the next S goes where P was
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  // ring units; of a Q tile: Q there, Q read; of a slot: S written, the first and
  // second half of P written; of a Q tile: O final, O read, a product with V
  // done (not where S's arrival says it), its turn to issue; items there, read; rows'
  // maxima and sums there, read; a unit of values with a sequence's end there
  uint64_t *full = bars, *empty = bars + C::kRing, *q_full = bars + 2 * C::kRing, *q_free = q_full + 2;
  uint64_t *s_full = q_free + 2, *p_full = s_full + 2, *o_full = p_full + 4,
           *o_free = o_full + 2, *pv_done = o_free + 2, *turn = pv_done + 2, *item_full = turn + 2,
           *item_free = item_full + 2, *ml_full = item_free + 2, *ml_free = ml_full + 2,
           *tail_full = ml_free + 2, *all_done = tail_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* state = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

  const PrefillArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kStore = C::kSoftmax, kLoad = kStore + 4, kMma = kLoad + 1, kPlan = kMma + kTiles;

  pdl_release();
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kLoad && lane == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kTiles);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_free + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + 2 * i, 4);  // the four softmax warps of a tile
      mbar_init(p_full + 2 * i + 1, 4);
      mbar_init(o_full + i, 1);
      mbar_init(o_free + i, 4);
      mbar_init(pv_done + i, 1);
      mbar_init(turn + i, 1);
      mbar_init(item_full + i, 1);
      mbar_init(item_free + i, 1 + kTiles + 4 + C::kSoftmax);  // every warp that reads items
      mbar_init(ml_full + i, 4);
      mbar_init(ml_free + i, 4);
    }
    mbar_init(tail_full, 1);
    mbar_init(all_done, kTiles);
    *state = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const uint32_t ring = smem_addr(smem + C::kOffRing), qs = smem_addr(smem);
  float2* sums = reinterpret_cast<float2*>(smem + C::kOffSums);
  bool ok = true;

  int seen = 0;  // items read
  auto read_item = [&](Item& it, bool one_lane) {
    const bool there = bar_wait(item_full + (seen & 1), (seen >> 1) & 1, state);
    ok = one_lane ? there : __all_sync(~0u, there);
    if (!ok) return false;
    const volatile int* from = reinterpret_cast<const volatile int*>(smem + C::kOffItem + (seen & 1) * 64);
    int* to = reinterpret_cast<int*>(&it);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) to[i] = from[i];
    if (!one_lane) __syncwarp();
    if (one_lane || lane == 0) mbar_arrive(item_free + (seen & 1));
    ++seen;
    return it.b >= 0;
  };
  if (warp >= kLoad) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
  if (warp == kPlan) {
    // ---- the items of this CTA, one ahead of their use, and their Q tiles, into L2 at
    // once and into shared memory when the tile before has been read ------------------
    int qn[kTiles] = {};  // Q tiles loaded
    Walk walk = walk_from_top(p);
    for (int round = 0; ok; ++round) {
      // long items first, dealt out there and back, so that the CTAs' sums are alike
      const int i = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      Item it;
      // heads fastest: the long items of all of them come first
      const int n = p.by_per(i), sub = i - n * p.by_per.d;
      it.b = -1;
      int t;
      if (walk_to(p, n, walk, &it.b, &t)) {
        const Span sp = span_of(a, it.b);
        it.split = p.by_heads(sub);
        it.q0 = sp.q0, it.nq = sp.nq, it.k0 = sp.k0, it.nk = sp.nk;
        it.first = t * kTiles * p.tpt;
        it.hq0 = (sub - it.split * p.heads) * p.hg;
        it.h = p.by_G(it.hq0);
        // the parts are equal numbers of tiles of the last Q tile's keys
        auto keys = [&](int queries) {
          const int last = min(queries, it.nq) - 1;
          return a.causal ? min(it.nk, it.nk - it.nq + last + 1) : it.nk;
        };
        const int most = keys(it.first + kTiles * p.tpt);
        int part = most > 0 ? (most + kKeys - 1) / kKeys : 0;
        if (p.splits > 1) part = (part + p.splits - 1) / p.splits;
        it.lo = it.split * part;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          it.keys[s] = keys(it.first + (s + 1) * p.tpt);
          const int n = it.first + s * p.tpt < it.nq && it.keys[s] > 0 ? (it.keys[s] + kKeys - 1) / kKeys : 0;
          it.n[s] = s < kTiles ? max(0, min(n, it.lo + part) - it.lo) : 0;
        }
      }
      if (seen >= 2)
        ok = __all_sync(~0u, bar_wait(item_free + (seen & 1), ((seen >> 1) - 1) & 1, state));
      if (!ok) break;
      if (lane == 0) {
        volatile int* to = reinterpret_cast<volatile int*>(smem + C::kOffItem + (seen & 1) * 64);
        const int* from = reinterpret_cast<const int*>(&it);
#pragma unroll
        for (int e = 0; e < (int)(sizeof(Item) / 4); ++e) to[e] = from[e];
        mbar_arrive(item_full + (seen & 1));
      }
      __syncwarp();
      ++seen;
      if (it.b < 0) break;
#pragma unroll
      for (int s = 0; s < kTiles; ++s) {
        if (it.n[s] == 0) continue;
        const int y = it.q0 + it.first + s * p.tpt;
        if (lane < D / 64) tma_3d_prefetch(&map_q, 64 * lane, it.hq0, y);
        if (qn[s] > 0) ok = ok && __all_sync(~0u, bar_wait(q_free + s, (qn[s] - 1) & 1, state));
        if (!ok) break;
        ++qn[s];
        if (lane == 0) {
          mbar_expect_tx(q_full + s, (uint32_t)(p.hg * p.tpt * D * 2));
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c)
            tma_3d(qs + s * C::kQ + c * kRows * 128, &map_q, 64 * c, it.hq0, y, q_full + s);
        }
        __syncwarp();
      }
    }
    for (int s = 0; s < kTiles; ++s)  // the copies land before the CTA ends
      if (qn[s] > 0) static_cast<void>(mbar_wait(q_full + s, (qn[s] - 1) & 1, nullptr));
  } else if (warp == kLoad) {
    // ---- loads: K and V tiles through the ring in the order of their use:
    // K_0 V_0 K_1 V_1 ..., or with one Q tile K_0 K_1 V_0 K_2 V_1 ... --------------
    int u = 0, tails = 0;  // units issued; those that waited for a sequence's end
    Item it;
    while (read_item(it, false)) {
      const int most = max(it.n[0], it.n[1]), key0 = it.k0 + it.lo * kKeys;
      const int clear_from = it.nk > kClear ? it.k0 + it.nk : 0x7fffffff;
#pragma unroll 1
      for (int i = 0; i < 2 * most && ok; ++i) {
        bool v = i & 1;
        int j = i / 2;
        if (kTiles == 1 && i > 0 && i < 2 * most - 1) v = !v, j = v ? j - 1 : j + 1;
#pragma unroll 1
        for (int k = 0; k < C::kUnits; ++k, ++u) {
          const int st = u % C::kRing, round = u / C::kRing, y = key0 + j * kKeys;
          if (round > 0) ok = __all_sync(~0u, bar_wait(empty + st, (round - 1) & 1, state));
          if (!ok) break;
          const uint32_t to = ring + st * C::kUnit;
          if (__builtin_expect(v && y + (k + 1) * C::kVKeys > clear_from, 0)) {
            const int at = y + k * C::kVKeys, left = it.k0 + it.nk - at;
            ok = load_tail<D>(&map_v, to, tail_full, tails & 1, full + st, it.h, at, left, state);
            if (!ok) break;
            tails += left > 0;
            continue;
          }
          if (elected()) {  // boxes of 64 columns: K by columns, V by keys
            mbar_expect_tx(full + st, C::kUnit);
            if (v) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_3d(to + c * C::kVKeys * 128, &map_v, 64 * c, it.h, y + k * C::kVKeys, full + st);
            } else {
#pragma unroll
              for (int c = 0; c < C::kCols / 64; ++c)
                tma_3d(to + c * kKeys * 128, &map_k, k * C::kCols + 64 * c, it.h, y, full + st);
            }
          }
          __syncwarp();
        }
      }
      if (!ok) break;
    }
    // whatever becomes of the MMAs, the copies land before the CTA ends
    for (int v = max(0, u - C::kRing); v < u; ++v)
      static_cast<void>(mbar_wait(full + v % C::kRing, (v / C::kRing) & 1, nullptr));
  } else if (warp >= kMma && warp < kMma + kTiles) {
    // ---- MMAs.  The warp stays converged and an elected lane issues each product
    // in straight-line code (an MMA costs the issue 110 clocks in a lane's own
    // branch, where its operands cannot be uniform registers, and the tensor core
    // 64).  The tensor core takes few MMAs ahead, so a pause in the issue is a
    // pause in the products: with two Q tiles each has an issuing warp of its own,
    // and one waits for barriers while the other's MMAs run -------------------------
    const int s = warp - kMma;
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && __all_sync(~0u, bar_wait(bar, phase & 1, state));
    };
    struct Place {  // in the ring
      int st;
      uint32_t phase;
    } next{0, 0};
    auto step = [&](Place& x) {
      if (++x.st == C::kRing) x.st = 0, x.phase ^= 1;
    };
    auto take = [&] {  // the next K or V tile's
      const Place x = next;
      for (int k = 0; k < C::kUnits; ++k) step(next);
      return x;
    };
    // of the items before: tiles of this Q tile, rounds of turns, outputs of this Q tile
    int done = 0, rounds = 0, outs = 0;
    Item it;
    while (read_item(it, false)) {
      const int tiles = s ? it.n[1] : it.n[0], theirs = s ? it.n[0] : it.n[1], most = max(tiles, theirs);
      if (most == 0) continue;
      auto slot_of = [&](int j) { return kTiles == 1 ? (done + j) & 1 : s; };
      auto use_of = [&](int j) { return kTiles == 1 ? (done + j) >> 1 : done + j; };
      // A K or V tile that the other Q tile does not use is released for both.
      auto release = [&](int j, int st) {
        mma_commit(empty + st);
        if (kTiles == 2 && j >= theirs) mma_commit(empty + st);
      };
      // S of tile j into its slot
      auto scores = [&](int j, Place at) {
        const int slot = slot_of(j);
        if (j == 0) wait(q_full + s, outs);
#pragma unroll
        for (int k = 0; k < C::kUnits; ++k) {  // by columns
          if (!kAfter || j == 0) wait(full + at.st, at.phase);
          fence_after();
          if (ok && elected()) {
            const uint32_t qd = tile_desc(qs + s * C::kQ + k * (C::kCols / 64) * kRows * 128, 16);
            const uint32_t kd = tile_desc(ring + at.st * C::kUnit, 16);
#pragma unroll
            for (int c = 0; c < C::kCols / 64; ++c)  // descriptors count 16 bytes
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int o = c * (kRows * 128 / 16) + 2 * e;
                if (k == 0 && c == 0 && e == 0)
                  mma_ss<false>(tmem + slot * kKeys, qd + o, kd + o, idesc<kKeys, false>());
                else
                  mma_ss<true>(tmem + slot * kKeys, qd + o, kd + o, idesc<kKeys, false>());
              }
            release(j, at.st);
            if (k == C::kUnits - 1) {
              mma_commit(s_full + slot);
              if (j == tiles - 1) mma_commit(q_free + s);
            }
          }
          __syncwarp();
          step(at);
        }
      };
      if (!kAfter) {
        const Place k = take();
        if (tiles > 0) scores(0, k);
      }
#pragma unroll 1
      for (int j = kAfter ? -1 : 0; j < most && ok; ++j) {
        const bool mine = j >= 0 && (kTiles == 1 || j < tiles), more = j + 1 < tiles;
        Place v{0, 0}, k{0, 0};  // V_j, K_(j + 1), in the order of the loads
        if (kTiles == 1 && j + 1 < most) k = take();
        if (j >= 0) v = take();
        if (kTiles == 2 && j + 1 < most) k = take();
        if (!kAfter && more) scores(j + 1, k);
        // O += P V, over the first and second 64 keys
        const int slot = slot_of(j), use = use_of(j);
        if (mine) {
          Place x = v;
#pragma unroll
          for (int k = 0; k < C::kUnits; ++k, step(x)) wait(full + x.st, x.phase);
          if (j == 0 && outs > 0) wait(o_free + s, outs - 1);
        }
        if (kAfter && j >= 0 && more) wait(full + k.st, k.phase);
#pragma unroll
        for (int half = 0; half < 2 && j >= 0; ++half) {
          if (mine) wait(p_full + 2 * slot + half, use);
          // Two Q tiles take turns: issued side by side their MMAs would alternate,
          // both S would arrive together and the tensor core would stand still
          // during both softmaxes (540 for 442 us, 8192 tokens).
          if (kAfter && half == 0) {
            const int t = rounds + j - (s == 0);
            if (t >= 0) wait(turn + s, t);
          }
          if (!mine) break;
          fence_after();
          if (ok && elected()) {
            const uint32_t pa = tmem + slot * kKeys + 32 * half;
            const uint32_t d = tmem + 2 * kKeys + s * D;
            const uint32_t vd = tile_desc(ring + v.st * C::kUnit + (C::kUnits == 2 ? 0 : 8192 * half),
                                          C::kVKeys * 128);
            if (half > 0 || j > 0)
              mma_ts<true>(d, pa, vd, idesc<D, true>());
            else
              mma_ts<false>(d, pa, vd, idesc<D, true>());
#pragma unroll
            for (int e = 1; e < 4; ++e)  // 16 keys: 8 columns of P, 2048 bytes of V
              mma_ts<true>(d, pa + 8 * e, vd + 128 * e, idesc<D, true>());
            if (half == 1 || C::kUnits == 2) release(j, v.st);
            if (half == 1) {
              if (kTiles == 1) mma_commit(pv_done + s);
              if (j == tiles - 1) mma_commit(o_full + s);
            }
          }
          __syncwarp();
          if (C::kUnits == 2) step(v);
        }
        if (kAfter && more) scores(j + 1, k);
        if (kAfter && j >= 0 && ok && lane == 0) mbar_arrive(turn + 1 - s);
      }
      if (!ok) break;
      done += tiles;
      rounds += most;
      outs += tiles > 0;
    }
    if (elected()) mma_commit(all_done);
    __syncwarp();
  } else if (warp < C::kSoftmax) {
    // ---- softmax: thread = row of Q tile s ------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int s = kTiles == 1 ? 0 : warp >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int row = 32 * quarter + lane;
    const float scale2 = a.scale * kLog2e;
    const uint32_t o_at = tmem + lanes + 2 * kKeys + s * D;
    // this row's token of the tile, and those of the warp's first and last row
    const int my_tok = p.by_hg(row), tok_lo = p.by_hg(32 * quarter), tok_hi = p.by_hg(32 * quarter + 31);
    int done = 0, outs = 0;  // tiles and items before this one
    Item it;
    while (read_item(it, false)) {
      const int first = it.first + s * p.tpt, tiles = s ? it.n[1] : it.n[0];
      // keys of this part that a row sees: this one, the warp's first and its last
      auto sees_of = [&](int t) {
        return (a.causal ? min(it.nk, it.nk - it.nq + first + t + 1) : it.nk) - it.lo * kKeys;
      };
      const int sees = sees_of(my_tok), least = sees_of(tok_lo), best = sees_of(tok_hi);
      float m = kNegInf;  // what P refers to, in units of log2
      bool ready = false;
      uint64_t sum2[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
      for (int j = 0; j < tiles && ok; ++j) {
        const int g = done + j, slot = kTiles == 1 ? g & 1 : s, use = kTiles == 1 ? g >> 1 : g;
        const uint32_t at = tmem + lanes + slot * kKeys;
        ok = __all_sync(~0u, ready || bar_wait(s_full + slot, use & 1, state));
        if (!ok) break;
        fence_after();
        const int left = sees - j * kKeys, left_lo = least - j * kKeys, left_hi = best - j * kKeys;
        if (__builtin_expect(left_lo < kKeys, 0)) {
          // Keys past what a row sees, in TMEM: a loop that fits the instruction cache
          // (short sequences are masked tiles for the most part).
#pragma unroll 1
          for (int c = left_lo < 32 ? 0 : left_lo & ~31; c < (left_hi > 64 ? kKeys : 64); c += 32) {
            uint32_t x[32];
            tmem_ld32(at + c, x);
            tmem_wait_ld();
            const int in = left - c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= in) x[e] = 0xff800000u;
            tmem_st32(at + c, x);
          }
          tmem_wait_st();
        }
        // The second 64 columns are read twice, for the maximum and again for their
        // exponentials: 128 values held beside P's do not fit the registers.
        uint32_t v[64];
        auto read_s = [&](uint32_t* to, int c0) {
          tmem_ld32(at + c0, to);
          tmem_ld32(at + c0 + 32, to + 32);
        };
        float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
        auto take_max = [&](const uint32_t* x) {
#pragma unroll
          for (int c = 0; c < 64; c += 2)
            top[c / 2 % 4] = max3(top[c / 2 % 4], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        };
        {
          uint32_t second[64];
          read_s(v, 0);
          read_s(second, 64);
          tmem_wait_ld();
          take_max(v);
          if (left_hi > 64) take_max(second);
        }
        const float t2 = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale2;
        if (j == 0) {
          m = t2;
        } else if (__builtin_expect(__any_sync(~0u, t2 > m + kSlack), 0)) {
          // O moves to the new maximum once the product with the tile before is
          // done (where S follows P, S says so)
          if constexpr (!kAfter) {
            ok = __all_sync(~0u, bar_wait(pv_done + s, (g - 1) & 1, state));
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
        auto half_p = [&](int half) {  // of v
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            unpair(fma2(pair(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), ss, zz), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum2[e & 1] = add2(sum2[e & 1], pair(x0, x1));
            x[e] = bf16x2(x0, x1);
          }
          tmem_st32(at + 32 * half, x);
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
          const int ng = g + 1, nslot = kTiles == 1 ? ng & 1 : s, nuse = kTiles == 1 ? ng >> 1 : ng;
          ready = j + 1 < tiles && mbar_test(s_full + nslot, nuse & 1);
        }
        if (left_hi > 64) {
          read_s(v, 64);
          tmem_wait_ld();
          half_p(1);
        } else {
          const uint32_t none[32] = {};
          tmem_st32(at + 32, none);
        }
        publish(1);
      }
      done += tiles;
      if (!ok) break;
      if (first >= it.nq) continue;

      // the rows' maxima and sums, for the warps that store
      float lo, hi;
      unpair(add2(sum2[0], sum2[1]), lo, hi);
      if (outs > 0) {
        ok = __all_sync(~0u, bar_wait(ml_free + s, (outs - 1) & 1, state));
        if (!ok) break;
      }
      ++outs;
      sums[s * kRows + row] = make_float2(m, lo + hi);
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_full + s);
    }
  } else if (warp < kLoad) {
    // ---- the output: O over its sum, while the next item is in work ---------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsStore));
    const int quarter = warp & 3, row = 32 * quarter + lane;
    const bool aligned32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0, parts = p.splits > 1;
    const int my_tok = p.by_hg(row), my_head = row - my_tok * p.hg;
    unsigned told = 0, outs = 0;  // bit s: parity of Q tile s's items, of its outputs
    Item it;
    while (read_item(it, false)) {
#pragma unroll 1
      for (int s = 0; s < kTiles; ++s) {
        const int first = it.first + s * p.tpt, tiles = s ? it.n[1] : it.n[0];
        if (first >= it.nq) break;
        const int tok = first + my_tok, hq = it.hq0 + my_head;
        const bool mine = row < p.hg * p.tpt && tok < it.nq;
        const int64_t out_row = (int64_t)(it.q0 + tok) * a.Hq + hq;
        ok = __all_sync(~0u, bar_wait(ml_full + s, (told >> s) & 1, state));
        if (!ok) break;
        told ^= 1u << s;
        const float2 ml = sums[s * kRows + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_free + s);
        const float l = ml.y;
        if (mine) {
          if (parts)
            p.ml[(int64_t)it.split * a.Tq * a.Hq + out_row] = ml;
          else if (a.lse)
            a.lse[out_row] = l == 0.0f ? kNegInf : (ml.x + __log2f(l)) * kLn2;
        }
        if (tiles > 0) {
          ok = __all_sync(~0u, bar_wait(o_full + s, (outs >> s) & 1, state));
          if (!ok) break;
          outs ^= 1u << s;
          fence_after();
        }
        uint64_t checked = pair(0.0f, 0.0f);
        if (tiles > 0 || !parts) {
          const uint32_t o_at = tmem + ((uint32_t)(32 * quarter) << 16) + 2 * kKeys + s * D;
          const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
          char* to = parts ? reinterpret_cast<char*>(p.part + ((int64_t)it.split * a.Tq * a.Hq + out_row) * D)
                           : reinterpret_cast<char*>(a.out + out_row * D);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            if (tiles > 0) {
              tmem_ld16(o_at + c, o);
              tmem_wait_ld();
            }
            if (l == 0.0f) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0u;
            }
            const uint64_t zero2 = pair(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 16; e += 2)  // 0 as long as every value is finite
              checked = fma2(pair(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), zero2, checked);
            if (!mine) continue;
            if (parts) {
              store32(to, o, true);
              store32(to + 32, o + 8, true);
              to += 64;
            } else {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float y0, y1;
                unpair(mul2(pair(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), pair(inv, inv)),
                       y0, y1);
                y[e] = bf16x2(y0, y1);
              }
              store32(to, y, aligned32);
              to += 32;
            }
          }
          if (tiles > 0) {  // the next item's product may come
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free + s);
          }
        }
        // rows whose sum is finite and whose output is not
        float lo, hi;
        unpair(checked, lo, hi);
        const unsigned again = __ballot_sync(~0u, mine && !(lo + hi == 0.0f) && l == l);
        if (again) {
          // the part's keys in the tiles, those past the sequence's end too unless they
          // were cleared
          const int key0 = it.lo * kKeys,
                    end = min(tiles * kKeys, (it.nk > kClear ? it.nk : (int)a.Tk - it.k0) - key0);
          const int sees = (a.causal ? min(it.nk, it.nk - it.nq + tok + 1) : it.nk) - key0;
          __syncwarp();
          repair<D>(p, it.split, again, it.q0 + tok, hq, min(sees, end), it.h, it.k0 + key0, end, state);
        }
      }
      if (!ok) break;
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(const_cast<int*>(state), kAborted);
    if (lane == 0) atomicOr(status, kDevTimeout);
  }
  if ((*state & kAborted) && warp == kMma && lane == 0) static_cast<void>(mbar_wait(all_done, 0, nullptr));
  fence_before();
  __syncthreads();
  if (warp == kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the parts of each row, in order: a warp a row, rows of the sequences.
template <int D>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(Args p) {
  constexpr int N = D / 32;
  pdl_release();
  pdl_wait();
  const PrefillArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.Tq * a.Hq, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int64_t t = row / a.Hq;
  if (t < clamped(__ldg(a.cu_q), a.Tq) || t >= clamped(__ldg(a.cu_q + a.B), a.Tq)) return;
  RowState<D> r;
  for (int i = 0; i < p.splits; ++i) {
    const float2 ml = p.ml[i * rows + row];
    if (ml.y == 0.0f) continue;  // a part without keys: its sums were not written
    float o[N];
    const float* from = p.part + (i * rows + row) * D + lane * N;
    if constexpr (N == 2) {
      const float2 v = *reinterpret_cast<const float2*>(from);
      o[0] = v.x, o[1] = v.y;
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + e);
        o[e] = v.x, o[e + 1] = v.y, o[e + 2] = v.z, o[e + 3] = v.w;
      }
    }
    r.join(ml.x, ml.y, o);
  }
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;
  if (a.lse && lane == 0) a.lse[row] = r.l == 0.0f ? kNegInf : r.m * kLn2 + logf(r.l);
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + row * D + lane * N + i) = bf16x2(r.o[i] * inv, r.o[i + 1] * inv);
}

constexpr int64_t kSms = 152;

// The heads of a Q tile: of the divisors of G, the one whose tiles of
// floor(128 / heads) tokens waste the fewest rows on sequences of the mean
// length (one sequence: on it; several: half a run each); the most heads where
// several do (fewer K and V loads a row).  Against one head a tile, five of
// 128: 16 prompts of 25 tokens 6.4 us for 15.4, of 550 68 for 91; one of 8192
// takes 450 either way.
int heads_of_tile(int64_t G, int64_t B, int64_t Tq, int tiles) {
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

struct Plan {
  int hg, tpt, splits;
  int64_t items, heads;
};

// Where the items fill less than half the SMs and the keys are long, each
// item's keys are cut into parts of at least eight tiles, for about one item an
// SM: 64 queries over 8192 keys, 8 x 5 heads of 128, take 28 us so and 90 whole.
// (An item costs about four tiles of its own: with 180 items of 18 to 28 tiles two
// parts took 84 us and one 78.)  A function of the shapes alone, so
// the workspace query and the launch agree.
Plan plan_of(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D) {
  Plan r;
  const int tiles = D == 256 ? 1 : 2;
  const int64_t G = Hq / Hkv;
  r.hg = heads_of_tile(G, B, Tq, tiles);
  r.tpt = kRows / r.hg;
  r.heads = Hkv * (G / r.hg);
  // every sequence has at most one run that is not whole
  const int64_t run = tiles * r.tpt;
  r.items = Tq / run + (B < Tq ? B : Tq);
  const int64_t likely = (B == 1 ? (Tq + run - 1) / run : r.items) * r.heads;
  const int64_t long_keys = B > 0 ? Tk / B / kKeys / 8 : 0;
  int64_t n = likely > 0 ? kSms / likely : 1;
  n = n < long_keys ? n : long_keys;
  r.splits = (int)(n < 2 ? 1 : n > 32 ? 32 : n);
  return r;
}

size_t workspace_of(const Plan& r, int64_t Tq, int64_t Hq, int64_t D) {
  return r.splits > 1 ? (size_t)r.splits * (size_t)(Tq * Hq) * (size_t)(D * 4 + 8) + 256 : 0;
}

template <int D>
cudaError_t launch(const PrefillArgs& a, void* ws, cudaStream_t st) {
  using C = Cfg<D>;
  const Plan plan = plan_of(a.B, a.Tq, a.Tk, a.Hq, a.Hkv, D);
  int64_t work;
  if (!mul_ok(plan.items, plan.heads * plan.splits, &work) || work > INT32_MAX / 2)
    return cudaErrorInvalidValue;
  const int G = (int)(a.Hq / a.Hkv);
  Args p{a, G, 0, 0, 0, Divider(plan.heads * plan.splits), Divider(plan.heads), Divider(G), Divider(plan.hg),
         Divider(C::kTiles * plan.tpt), 1, 0, nullptr, nullptr};
  p.hg = plan.hg;
  p.tpt = plan.tpt;
  p.splits = plan.splits;
  p.part = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~(uintptr_t)255);
  p.ml = reinterpret_cast<float2*>(p.part + (size_t)plan.splits * a.Tq * a.Hq * D);
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
  p.heads = (int)plan.heads;
  const int64_t steps = (a.B + 31) / 32;  // of one way
  p.ways = steps < kSteps ? (int)(kSteps / steps) : 1;
  e = launch_pdl(kern, dim3((unsigned)(work < kSms ? work : kSms)), dim3(C::kThreads), C::kSmem, st,
                 mq, mk, mv, p, status);
  if (e != cudaSuccess || plan.splits == 1) return e;
  return launch_pdl(attn_prefill_join_kernel<D>, dim3((unsigned)((a.Tq * a.Hq + 7) / 8)), dim3(256), 0,
                    st, p);
}

}  // namespace

size_t attn_prefill_workspace(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Tq == 0) return 0;
  return workspace_of(plan_of(B, Tq, Tk, Hq, Hkv, D), Tq, Hq, D);
}

cudaError_t launch_attn_prefill(const PrefillArgs& a, void* ws, cudaStream_t st) {
  switch (a.D) {
    case 64: return launch<64>(a, ws, st);
    case 128: return launch<128>(a, ws, st);
    default: return launch<256>(a, ws, st);
  }
}

}  // namespace ptq
