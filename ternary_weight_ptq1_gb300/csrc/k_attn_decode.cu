// k_attn_decode.cu -- attention of one new token of each sequence over its
// paged key-value cache.
//
//   s_j = scale q . k_j,  p_j = 2^(s_j log2(e) - m),  out = sum_j p_j v_j / sum_j p_j
//
// Every cached byte is read once for all the query heads that share it, so
// HBM bounds the operator: 2 head_dim bytes (int8, plus two scales) or
// 4 head_dim bytes a token and kv head.  A tile of 32 tokens is about 900
// instructions of a warp, so issue is busy for half of the time at the full
// rate; few or short sequences are bound by a call's chain of latencies
// (lengths, page numbers, rows, the joins).
//
// Measured in CUDA graphs: 64 sequences of up to 8192 tokens, 8 x 8 heads of 128, bf16
// over int8, in 104 us (5.5 TB/s, 82% of the copy rate); one of 131,001 tokens, 4 x 6
// of 256, bf16 cache, in 89 us (6.0 TB/s, 89%); 96 of up to 700 tokens, 16 heads
// of 64, bf16, in 31 us (59%: three starts a CTA); 8 of up to 4096, 8 x 5 of 128,
// fp32 over int8, in 14.4 us; one of 777 tokens, fp32 over bf16, in 8.7 us.
//
// Split.  The tokens of one (sequence, kv head) are cut into tiles of kT; the
// tiles of all of them, in order, are dealt to the CTAs in runs of equal cost,
// so ragged batches keep every SM busy to the end whatever the lengths are.
// (The start and end of a (sequence, kv head) cost as much as kLead tiles:
// without them the CTA that got the shortest sequences of a ragged batch took
// three times as long as the others: 92 us for 36 on 96 sequences of up to 700
// tokens.)  The lengths are on the device: each CTA
// adds them up itself.  The part of a (sequence, kv head) inside one CTA's run
// is a segment; a segment that is a whole (sequence, kv head) writes its
// output, the others write their maximum, sum and output sums to the workspace
// and a second kernel joins them in order.  Where the sequences are few and
// short, a cluster of CTAs shares each (sequence, kv head) instead and joins
// its parts through distributed shared memory, in one launch.
//
// Inside a CTA each warp owns its tiles alone: it copies them into a ring of
// its own in shared memory (cp.async, the copies of the next tiles always in
// flight, across segments too), keeps its own maximum, sum and output in
// registers, and meets the other warps only at the end of a segment.
//
// Arithmetic.  Both products run on the 16 x 8 x 16 matrix instruction with
// fp32 sums.  It takes 16-bit factors: int8 codes are exact in fp16 and bf16
// rows are exact as they are, so only q and p are split, into two terms.  The
// instruction's rows 0-7 hold the first terms of eight query heads, rows 8-15
// the second, and the two rows' results are added (a kv head has rarely more
// than eight query heads, so the second terms cost no instruction):
//   int8 cache: two fp16 terms, 22 bits (q scaled by a power of two to its
//     row's largest value, p times its value's scale by the largest such product
//     of the row so far: a value of great scale and no weight costs the others no
//     bits);
//   bf16 cache, bf16 q: q is exact, p has two bf16 terms, 16 bits;
//   bf16 cache, fp32 q: three bf16 terms, the third in a second instruction.
// More than eight heads take two row blocks a warp (kBlocks) up to head_dim
// 128 (64 x 4096 tokens, 2 x 16 heads of 128: 52 us over int8 and 57 over bf16,
// for 63 and 89 with a block each); where there are more blocks still, each
// reads the cache again (the same moment, so mostly from L2).
// The fp32 routes, those of two row blocks and 256-wide heads over int8 (64 x 4096
// tokens, 4 x 6 heads: 123 us for 129) add each tile's product to the output in
// fp32 registers; the others let the matrix unit accumulate, whose sums are rounded
// below the bf16 output's own rounding.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "attn_row.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kSms = 152;
constexpr int kWarps = 4;
constexpr int kLead = 16;
constexpr float kTiny = 1.2037062152420224e-35f;  // 2^-116, the smallest reference weight
constexpr float kPScale = 1024.0f;               // fp16 probabilities are stored times this

template <Act T, int D, bool kI8, int kBlocks>
struct Cfg {
  static constexpr int kT = kI8 || D == 64 ? 32 : 16;  // tokens of a tile
  static constexpr int kRow = D * (kI8 ? 1 : 2);       // bytes of a cached row
  static constexpr int kChunks = kRow / 16;            // 16-byte pieces of a row
  static constexpr int kTile = kT * kRow;
  static constexpr int kStage = 2 * kTile + (kI8 ? 2 * kT * 4 : 0);
  static constexpr int kStages = 2;
  static constexpr bool kThree = T == Act::F32 && !kI8;
  static constexpr bool kExactQ = T == Act::BF16 && !kI8;  // q's second terms are 0
  static constexpr bool kFresh = T == Act::F32 || kBlocks > 1 || (kI8 && D == 256);
  static constexpr int kHeads = 8 * kBlocks;            // query heads a warp serves
  static constexpr int kQ = kBlocks * D / 16 * 32 * 16;  // bytes of the query's fragments
  static constexpr int kOffQ3 = kWarps * kStages * kStage;
  static constexpr int kOffQ = kOffQ3 + (kThree ? kQ / 2 : 0);
  static constexpr int kOffF = kOffQ + kQ;              // score factor of each head
  static constexpr int kOffMl = kOffF + 16 * 4;         // (m, l) of each warp and head
  static constexpr int kOffBad = kOffMl + kWarps * 16 * 8;
  static constexpr int kOffScan = kOffBad + kWarps * kStages * 4;
  static constexpr int kOffPart = (kOffScan + 2 * kWarps * 8 + 32 + 15) / 16 * 16;  // (m, l) of each head
  static constexpr int kSmem = kOffPart + 16 * 8;
  static constexpr int kFit = (227 * 1024) / (kSmem + 1024);
  // CTAs of an SM: two keep HBM busy (64 x 4096 tokens, 8 x 8 heads of 128, bf16
  // cache: 164 us for 173 with three); at head_dim 64 the starts of short
  // sequences count more (96 x 350 tokens, 16 heads: 31.7 us with three for 34.7).
  static constexpr int kWish = D == 64 && kBlocks == 1 ? 3 : 2;
  static constexpr int kPerSm = kFit < 1 ? 1 : kFit > kWish ? kWish : kFit;
  // a warp's output (kHeads rows of fp32) is handed over in a stage, a cluster's
  // CTA's where the query's fragments were
  static_assert(kStage >= kHeads * D * 4 && kQ >= kHeads * D * 4, "room for an output");
};

constexpr int kMaxCtas = 3 * kSms;
constexpr int kCluster = 8;  // CTAs of a cluster

// Workspace: for each CTA two segments (one that began before its run, one
// that goes on after it), each kHeads rows of D sums, then their (m, l), then
// a note for the second kernel.
struct Note {
  int b, vh, last;  // the segment that goes on: its place, and the CTA that ends it; b = -1: none
  int pad;
};

struct Args {
  DecodeArgs a;
  float* part;    // [2 ctas][heads][D]
  float2* ml;     // [2 ctas][heads]
  Note* note;     // [ctas]
  int G, VH, HC;  // query heads of a kv head; row blocks in all, of one kv head
  bool whole;     // pages hold whole tiles (64 x 4096 tokens, 8 x 8 heads of 128 over int8: 100 us
                  // for 108 by rows)
  int cluster;    // CTAs of a (sequence, row block); 0: runs
};

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two of the four int8 codes of x ^ 0x80808080 as fp16: the byte c + 128
// under the exponent of 1024 is 1152 + c, and the difference is exact.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes(uint32_t x) {
  const uint32_t w = __byte_perm(x, 0x64646464u, kSel), base = 0x64806480u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&base));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// x0, x1 as a pair of 16-bit values, and what the rounding left.
template <bool kF16>
__device__ __forceinline__ uint32_t round2(float& x0, float& x1) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(x0, x1);
    x0 -= __low2float(h);
    x1 -= __high2float(h);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    x0 -= __low2float(h);
    x1 -= __high2float(h);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sums of the first and the second terms; an infinite value's second
// product may be infinite the other way (kInf: values may be infinite).
template <bool kInf>
__device__ __forceinline__ float both(float first, float second) {
  return kInf && !(fabsf(first) < __int_as_float(0x7f800000)) ? first : first + second;
}

// 1 / sum; a row whose scores are all -infinity is one that sees no key.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

__device__ __forceinline__ int length(const DecodeArgs& a, int b) {
  const int64_t most = a.table_width * a.c.page_tokens;
  const int n = __ldg(a.lens + b);
  return n < 0 ? 0 : n > most ? (int)most : n;
}

template <int kT>
__device__ __forceinline__ int tiles_of(int len) {
  return (int)(((unsigned)len + kT - 1) / kT);
}

// The units a (sequence, row block) of n tiles is dealt out in: kLead units for
// its start, then its tiles.
__device__ __forceinline__ int units(int n) { return n ? n + kLead : 0; }

// The part of one (sequence, row block) inside a CTA's run: tiles t0 .. t1 - 1
// of n.  b < 0: past the end of the run.
struct Segment {
  int b, vh, t0, t1, n, len;
  int64_t u;  // its first unit's place among all
};

// The tiles of the segment's (sequence, row block) in units [u0, u1); false: none.
__device__ __forceinline__ bool clip(Segment& s, int64_t u0, int64_t u1) {
  s.t0 = (int)max((int64_t)0, u0 - s.u - kLead);
  s.t1 = (int)min((int64_t)s.n, u1 - s.u - kLead);
  return s.t0 < s.t1;
}

template <int kT>
__device__ __forceinline__ void next_segment(Segment& s, const Args& p, int64_t u1) {
  s.u += units(s.n);
  s.t0 = s.t1 = 0;
  if (s.u >= u1) {
    s.b = -1;
    return;
  }
  if (++s.vh == p.VH) {
    s.vh = 0;
    do s.len = length(p.a, ++s.b);
    while (s.len == 0);
    s.n = tiles_of<kT>(s.len);
  }
  if (!clip(s, s.u, u1)) s.b = -1;  // the run ends before its first tile
}

template <Act T>
__device__ __forceinline__ void store_out4(void* out, int64_t e, float4 v) {
  if constexpr (T == Act::F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + e) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + e) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

__device__ __forceinline__ uint32_t peer(uint32_t at, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_ld2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// The weight of a part with maximum m and sum l in a whole with maximum top.
// l = 0: the part has no key.  m = -inf with l != 0: its scores are NaN.
__device__ __forceinline__ float part_weight(float2 ml, float top) {
  return ml.y == 0.0f ? 0.0f : ml.x == kNegInf ? 1.0f : exp2f(ml.x - top);
}

template <Act T, int D, bool kI8, int kBlocks>
__global__ void __launch_bounds__(kWarps * 32, Cfg<T, D, kI8, kBlocks>::kPerSm)
    attn_decode_kernel(Args p) {
  using C = Cfg<T, D, kI8, kBlocks>;
  constexpr int kT = C::kT, kNS = kT / 8, kNO = D / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const DecodeArgs& a = p.a;
  const int ps = (int)a.c.page_tokens, heads = (int)a.c.kv_heads;
  pdl_release();
  pdl_wait();

  // ---- the run of this CTA ---------------------------------------------------------
  int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kOffScan);  // [2][kWarps]
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)  // no key: 0 and -infinity
    if (length(a, b) == 0) {
      for (int64_t e = 4 * tid; e < a.Hq * D; e += 4 * kWarps * 32)
        store_out4<T>(a.out, b * a.Hq * D + e, make_float4(0.f, 0.f, 0.f, 0.f));
      if (a.lse)
        for (int64_t h = tid; h < a.Hq; h += kWarps * 32) a.lse[b * a.Hq + h] = kNegInf;
    }
  Segment seg{-1, 0, 0, 0, 0, 0, 0};
  int64_t u1 = 1, per = 1;
  if (p.cluster) {  // an equal part of this cluster's (sequence, row block)
    const int id = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    seg.vh = id % p.VH;
    seg.len = length(a, id / p.VH);
    seg.n = tiles_of<kT>(seg.len);
    seg.t0 = (int)((int64_t)seg.n * rank / p.cluster);
    seg.t1 = (int)((int64_t)seg.n * (rank + 1) / p.cluster);
    if (seg.n == 0) return;  // the whole cluster
    if (seg.t0 < seg.t1) seg.b = id / p.VH;
  } else {
    int64_t mine = 0;
    for (int b = tid; b < a.B; b += kWarps * 32) mine += units(tiles_of<kT>(length(a, b)));
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mine += __shfl_xor_sync(~0u, mine, i);
    if (lane == 0) scan[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += scan[w];
    total *= p.VH;
    // runs of equal cost, of whole rounds of the CTA's warps
    per = (total + gridDim.x - 1) / gridDim.x;
    per = (per + kWarps - 1) / kWarps * kWarps;
    const int64_t u0 = blockIdx.x * per;
    u1 = min(u0 + per, total);
    if (tid == 0) p.note[blockIdx.x] = Note{-1, 0, 0, 0};
    if (u0 >= total) return;
    // the sequence that holds unit u0: sequences are added up kWarps * 32 at a time
    int* found = reinterpret_cast<int*>(scan + 2 * kWarps);
    if (tid == 0) *found = -1;
    for (int64_t b0 = 0, base = 0;; b0 += kWarps * 32) {
      const int64_t b = b0 + tid;
      const int n = b < a.B ? units(tiles_of<kT>(length(a, (int)b))) : 0;
      int64_t incl = (int64_t)n * p.VH;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, incl, i);
        if (lane >= i) incl += o;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      int64_t before = base, all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
      }
      const int64_t end = before + incl, start = end - (int64_t)n * p.VH;
      if (u0 >= start && u0 < end) {
        *found = (int)b;
        scan[kWarps] = start;
      }
      base += all;
      if (u0 < base) break;
    }
    __syncthreads();
    {
      seg.b = *found;
      const int64_t in = u0 - scan[kWarps];
      seg.len = length(a, seg.b);
      seg.n = tiles_of<kT>(seg.len);
      seg.vh = (int)(in / units(seg.n));
      seg.u = scan[kWarps] + (int64_t)seg.vh * units(seg.n);
      // (a run that ends within its first kLead units has no tile)
      if (!clip(seg, u0, u1)) seg.b = -1;
    }
  }

  const int mine_tiles = seg.b < 0 ? 0 : seg.t1 - seg.t0;

  // ---- the ring --------------------------------------------------------------------
  unsigned char* ring = smem + warp * C::kStages * C::kStage;
  const uint32_t ring_at = smem_at(ring);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::kOffBad) + warp * C::kStages;
  Segment ahead = seg;
  int at = ahead.t0 + warp;
  auto settle = [&] {  // `at` to this warp's next tile of the run
    while (ahead.b >= 0 && at >= ahead.t1) {
      next_segment<kT>(ahead, p, u1);
      at = ahead.t0 + warp;
    }
  };
  settle();
  // where this lane's piece (16 bytes) of a group of 32 pieces goes: the piece's
  // place in its row is exchanged by row, so that eight rows read together use
  // different banks
  auto place = [&](int i) {
    const int r = (i * 32 + lane) / C::kChunks, c = lane % C::kChunks;
    return (uint32_t)(r * C::kRow + ((c ^ (C::kChunks >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
  };
  auto prefetch = [&](int stage) {
    if (ahead.b >= 0) {
      const uint32_t dst = ring_at + stage * C::kStage;
      const int32_t* pages = a.table + ahead.b * a.table_width;
      const int j0 = at * kT, head = ahead.vh / p.HC;
      if (p.whole && ahead.len - j0 >= kT) {  // a tile inside one page: one stretch of rows
        const int page = __ldg(pages + (unsigned)j0 / (unsigned)ps);
        const bool in = (unsigned)page < (unsigned)a.c.pages;
        if (lane == 0) bad[stage] = !in;
        const int64_t row = ((int64_t)(in ? page : 0) * heads + head) * ps + (unsigned)j0 % (unsigned)ps;
        const char* k = static_cast<const char*>(a.c.k) + row * C::kRow + lane * 16;
        const char* v = static_cast<const char*>(a.c.v) + row * C::kRow + lane * 16;
#pragma unroll
        for (int i = 0; i < kT * C::kChunks / 32; ++i) {
          copy16(dst + place(i), k + i * 512, true);
          copy16(dst + place(i) + C::kTile, v + i * 512, true);
        }
        if constexpr (kI8) {
          copy4(dst + 2 * C::kTile + 4 * lane, a.c.k_scale + row + lane, true);
          copy4(dst + 2 * C::kTile + 4 * kT + 4 * lane, a.c.v_scale + row + lane, true);
        }
      } else {
        const unsigned j = (unsigned)j0 + lane % kT;
        int64_t row = -1;
        bool wrong = false;
        if (lane % kT < ahead.len - j0) {
          const int page = __ldg(pages + j / (unsigned)ps);
          wrong = (unsigned)page >= (unsigned)a.c.pages;
          if (!wrong) row = ((int64_t)page * heads + head) * ps + j % (unsigned)ps;
        }
        const uint32_t any = __ballot_sync(~0u, wrong);
        if (lane == 0) bad[stage] = any;
#pragma unroll
        for (int i = 0; i < kT * C::kChunks / 32; ++i) {
          const int64_t src = __shfl_sync(~0u, row, (i * 32 + lane) / C::kChunks);
          const int64_t off = (src < 0 ? 0 : src) * C::kRow + lane % C::kChunks * 16;
          copy16(dst + place(i), static_cast<const char*>(a.c.k) + off, src >= 0);
          copy16(dst + place(i) + C::kTile, static_cast<const char*>(a.c.v) + off, src >= 0);
        }
        if constexpr (kI8) {
          const int64_t off = row < 0 ? 0 : row;
          copy4(dst + 2 * C::kTile + 4 * lane, a.c.k_scale + off, row >= 0);
          copy4(dst + 2 * C::kTile + 4 * kT + 4 * lane, a.c.v_scale + off, row >= 0);
        }
      }
      at += kWarps;
      settle();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < C::kStages - 1; ++i) prefetch(i);
  int stage = C::kStages - 1;  // the stage used last (none yet): free

  uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQ);
  uint2* q3 = reinterpret_cast<uint2*>(smem + C::kOffQ3);
  float* qfac = reinterpret_cast<float*>(smem + C::kOffF);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);

  while (seg.b >= 0) {
    const int h0 = (seg.vh / p.HC) * p.G, r0 = (seg.vh % p.HC) * C::kHeads;
    const int rows = min(p.G - r0, C::kHeads);  // query heads of this block
    // ---- the query's fragments -----------------------------------------------------
    // Element d of head r: half a word of lane 4 (r % 8) + t of step d / 16, word
    // 2 hi of its first term and 2 hi + 1 of its second.  The int8 rows are read as
    // 16-byte chunks whose bytes 4 t .. 4 t + 3 a lane holds, so its four k are
    // those d.
    for (int r = warp; r < C::kHeads; r += kWarps) {
      constexpr int N = D / 32;
      float x[N];
      const int64_t e = seg.b * a.q_stride + (int64_t)(h0 + r0 + r) * D + lane * N;
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] = r >= rows ? 0.0f
               : T == Act::F32
                   ? __ldg(static_cast<const float*>(a.q) + e + i)
                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.q) + e + i) << 16);
      float f = a.scale * kLog2e;
      if constexpr (kI8) {  // to a largest magnitude in [2^11, 2^12)
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, i));
        int ex = m > 0.0f && m < __int_as_float(0x7f800000) ? ilogbf(m) - 11 : 0;
        ex = max(ex, -126);  // a row of subnormals only: still a normal factor
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = ldexpf(x[i], -ex);
        f *= ldexpf(1.0f, ex);
      }
      if (lane == 0) qfac[r] = f;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const int d = lane * N + i, dd = d % 16;
        const int t = kI8 ? dd / 4 : dd % 8 / 2, hi = kI8 ? dd / 2 % 2 : dd / 8;
        const int at_lane = ((r >> 3) * (D / 16) + d / 16) * 32 + (r & 7) * 4 + t;
        uint32_t* w = reinterpret_cast<uint32_t*>(qf + at_lane);
        w[2 * hi] = round2<kI8>(x[i], x[i + 1]);
        w[2 * hi + 1] = round2<kI8>(x[i], x[i + 1]);
        if constexpr (C::kThree)
          reinterpret_cast<uint32_t*>(q3 + at_lane)[hi] = round2<kI8>(x[i], x[i + 1]);
      }
    }
    __syncthreads();
    {  // the next segment's query rows, into L2
      Segment nx = seg;
      next_segment<kT>(nx, p, u1);
      constexpr int kBytes = D * (T == Act::F32 ? 4 : 2);
      if (nx.b >= 0 && tid < C::kHeads * (kBytes / 128)) {
        const int r = (nx.vh % p.HC) * C::kHeads + tid / (kBytes / 128);
        if (r < p.G) {
          const char* q = static_cast<const char*>(a.q) +
                          (nx.b * a.q_stride + (int64_t)((nx.vh / p.HC) * p.G + r) * D) * (kBytes / D);
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + tid % (kBytes / 128) * 128));
        }
      }
    }

    // head 8 h + g of the block: its maximum and sum so far, and its output
    // (first terms' rows, and without kFresh the second terms' rows apart)
    float fac[kBlocks], m[kBlocks], l[kBlocks];
    float ref[kBlocks];  // (int8) power of two above every p times value scale so far, p as m is now
    float o[kBlocks][kNO][C::kFresh ? 2 : 4] = {};
#pragma unroll
    for (int h = 0; h < kBlocks; ++h) {
      fac[h] = qfac[8 * h + g];
      m[h] = kNegInf;
      l[h] = 0.0f;
      ref[h] = kTiny;
    }

    for (int tile = seg.t0 + warp; tile < seg.t1; tile += kWarps) {
      const int free_stage = stage;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      prefetch(free_stage);
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
      __syncwarp();
      const uint32_t kt = ring_at + stage * C::kStage, vt = kt + C::kTile;
      const float* ks = reinterpret_cast<const float*>(ring + stage * C::kStage + 2 * C::kTile);
      const float* vs = ks + kT;

      // ---- scores ------------------------------------------------------------------
      float s[kBlocks][kNS][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint4 q[kBlocks];
        uint2 q2[kBlocks];
#pragma unroll
        for (int h = 0; h < kBlocks; ++h) {
          q[h] = qf[(h * (D / 16) + k) * 32 + lane];
          if constexpr (C::kThree) q2[h] = q3[(h * (D / 16) + k) * 32 + lane];
        }
        if constexpr (kI8) {  // four token groups of one 16-byte chunk
          uint32_t b[4];
          ldsm4(b, kt + lane * C::kRow + ((k ^ (C::kChunks >= 8 ? lane & 7 : (lane >> 1) & 3)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = b[i] ^ 0x80808080u, b0 = codes<0x4140>(x), b1 = codes<0x4342>(x);
#pragma unroll
            for (int h = 0; h < kBlocks; ++h)
              mma<true>(s[h][i], q[h].x, q[h].y, q[h].z, q[h].w, b0, b1);
          }
        } else {  // two token groups of two chunks
#pragma unroll
          for (int i = 0; i < kNS; i += 2) {
            const int r = 8 * i + (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm4(b, kt + r * C::kRow + ((c ^ (r & 7)) << 4));
#pragma unroll
            for (int h = 0; h < kBlocks; ++h) {
              mma<false>(s[h][i], q[h].x, q[h].y, q[h].z, q[h].w, b[0], b[1]);
              mma<false>(s[h][i + 1], q[h].x, q[h].y, q[h].z, q[h].w, b[2], b[3]);
              if constexpr (C::kThree) {
                mma<false>(s[h][i], q2[h].x, 0u, q2[h].y, 0u, b[0], b[1]);
                mma<false>(s[h][i + 1], q2[h].x, 0u, q2[h].y, 0u, b[2], b[3]);
              }
            }
          }
        }
      }

      // ---- softmax: column 2 t4 + i of group n is token 8 n + 2 t4 + i -------------
      const int left = seg.len - tile * kT;  // tokens of the tile that exist, if under kT
      // p as the second product's A: tokens 16 k .. + 15 are groups 2 k, 2 k + 1
      uint32_t ph[kBlocks][kNS][2], p3[kBlocks][C::kThree ? kNS : 1];
      float fade[kBlocks];
#pragma unroll
      for (int h = 0; h < kBlocks; ++h) {
        float x = kNegInf;
#pragma unroll
        for (int n = 0; n < kNS; ++n) {
          float c0 = fac[h], c1 = fac[h];
          if constexpr (kI8) {
            const float2 c = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * t4);
            c0 *= c.x, c1 *= c.y;
          }
          if constexpr (C::kExactQ) {
            s[h][n][0] *= c0;
            s[h][n][1] *= c1;
          } else {
            s[h][n][0] = (s[h][n][0] + s[h][n][2]) * c0;
            s[h][n][1] = (s[h][n][1] + s[h][n][3]) * c1;
          }
          if (left < kT) {
            if (8 * n + 2 * t4 >= left) s[h][n][0] = kNegInf;
            if (8 * n + 2 * t4 + 1 >= left) s[h][n][1] = kNegInf;
          }
          x = fmaxf(x, fmaxf(s[h][n][0], s[h][n][1]));
        }
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
        const float top = fmaxf(m[h], x), z = top == kNegInf ? 0.0f : top;
        const float f = exp2_fast(m[h] - z);
        m[h] = top;
        l[h] *= f;
        fade[h] = f;
        float inv = 1.0f, most = 0.0f;
#pragma unroll
        for (int n = 0; n < kNS; ++n) {
          float &e0 = s[h][n][0], &e1 = s[h][n][1];
          e0 = exp2_fast(e0 - z), e1 = exp2_fast(e1 - z);
          l[h] += e0 + e1;
          if constexpr (kI8) {
            const float2 w = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * t4);
            e0 *= w.x, e1 *= w.y;
            most = fmaxf(most, fmaxf(e0, e1));
          }
        }
        if constexpr (kI8) {
          // The reference moves with m, down too, and up to the tile's largest weight,
          // to 2^126 at most (larger weights still fit fp16; NaN stays in the products).
          most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
          most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
          const float old = ref[h] * f;  // (0 where the weights so far are nothing)
          const float up = fmaxf(fmaxf(most, 0.5f * kTiny), 0.5f * old);
          const uint32_t bits = (min(__float_as_uint(up), 0x7e000000u) & 0x7f800000u) + 0x00800000u;
          const float over = __uint_as_float(0x7f000000u - bits);  // one over it
          fade[h] = old * over;          // at most 2; the references alone may be 2^242 apart
          ref[h] = __uint_as_float(bits);
          inv = kPScale * over;
        }
#pragma unroll
        for (int n = 0; n < kNS; ++n) {
          float e0 = s[h][n][0], e1 = s[h][n][1];
          if constexpr (kI8) e0 *= inv, e1 *= inv;
          ph[h][n][0] = round2<kI8>(e0, e1);
          ph[h][n][1] = round2<kI8>(e0, e1);
          if constexpr (C::kThree) p3[h][n] = round2<kI8>(e0, e1);
        }
        if (bad[stage] != 0) l[h] = __int_as_float(0x7fc00000);  // a page outside the cache
      }

      // ---- output --------------------------------------------------------------------
      if constexpr (!C::kFresh) {
        if (__any_sync(~0u, fade[0] != 1.0f)) {
#pragma unroll
          for (int n = 0; n < kNO; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[0][n][e] *= fade[0];
        }
      }
      // kPer column groups at a time: 32 (int8) or 16 columns
      constexpr int kPer = kI8 ? 4 : 2;
#pragma unroll
      for (int n = 0; n < kNO; n += kPer) {
        float acc[kBlocks][kPer][4];
#pragma unroll
        for (int h = 0; h < kBlocks; ++h)
#pragma unroll
          for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (C::kFresh)
                acc[h][i][e] = 0.0f;
              else
                acc[h][i][e] = o[h][n + i][e];
            }
#pragma unroll
        for (int k = 0; k < kT / 16; ++k) {
          const int r = 16 * k + ((lane >> 3) & 1) * 8 + (lane & 7);
          const int c = (kI8 ? n / 2 : n) + (lane >> 4);
          uint32_t b[4];
          ldsm4t(b, vt + r * C::kRow + ((c ^ (C::kChunks >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
          if constexpr (kI8) {
            // bytes 0 and 2 of a word are the even column of two tokens, 1 and 3 the odd one
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] ^= 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = i & 1 ? codes<0x4341>(b[i & 2]) : codes<0x4240>(b[i & 2]);
              const uint32_t b1 = i & 1 ? codes<0x4341>(b[(i & 2) + 1]) : codes<0x4240>(b[(i & 2) + 1]);
#pragma unroll
              for (int h = 0; h < kBlocks; ++h)
                mma<true>(acc[h][i], ph[h][2 * k][0], ph[h][2 * k][1], ph[h][2 * k + 1][0],
                          ph[h][2 * k + 1][1], b0, b1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int h = 0; h < kBlocks; ++h) {
                mma<false>(acc[h][i], ph[h][2 * k][0], ph[h][2 * k][1], ph[h][2 * k + 1][0],
                           ph[h][2 * k + 1][1], b[2 * i], b[2 * i + 1]);
                if constexpr (C::kThree)
                  mma<false>(acc[h][i], p3[h][2 * k], 0u, p3[h][2 * k + 1], 0u, b[2 * i], b[2 * i + 1]);
              }
          }
        }
#pragma unroll
        for (int h = 0; h < kBlocks; ++h)
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if constexpr (C::kFresh) {
              o[h][n + i][0] = fmaf(o[h][n + i][0], fade[h], both<C::kExactQ>(acc[h][i][0], acc[h][i][2]));
              o[h][n + i][1] = fmaf(o[h][n + i][1], fade[h], both<C::kExactQ>(acc[h][i][1], acc[h][i][3]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[h][n + i][e] = acc[h][i][e];
            }
          }
      }
      __syncwarp();
    }

    // ---- the warps' parts of the segment ----------------------------------------------
    // Handed over in each warp's free stage, rows of D floats, 16-byte pieces
    // exchanged by row so that neighbouring rows use other banks.
    float* mine_o = reinterpret_cast<float*>(ring + stage * C::kStage);
#pragma unroll
    for (int h = 0; h < kBlocks; ++h) {
      const float back = kI8 ? ref[h] / kPScale : 1.0f;
      l[h] += __shfl_xor_sync(~0u, l[h], 1);
      l[h] += __shfl_xor_sync(~0u, l[h], 2);
      const int r = 8 * h + g;
      if (r >= rows) continue;
      if (t4 == 0) ml[warp * 16 + r] = make_float2(m[h], l[h]);
      auto col = [&](int n, int e) {
        if constexpr (C::kFresh)
          return o[h][n][e] * back;
        else
          return both<C::kExactQ>(o[h][n][e], o[h][n][e + 2]) * back;
      };
      if constexpr (kI8) {  // columns 16 c + 4 t4 .. + 3
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4*>(mine_o + r * D + (((4 * c + t4) ^ (r & 7)) << 2)) =
              make_float4(col(2 * c, 0), col(2 * c + 1, 0), col(2 * c, 1), col(2 * c + 1, 1));
      } else {  // columns 8 n + 2 t4, + 1
#pragma unroll
        for (int n = 0; n < kNO; ++n)
          *reinterpret_cast<float2*>(mine_o + r * D + (((2 * n + (t4 >> 1)) ^ (r & 7)) << 2) +
                                     2 * (t4 & 1)) = make_float2(col(n, 0), col(n, 1));
      }
    }
    // where each warp's part is
    int* where = reinterpret_cast<int*>(scan);
    if (lane == 0) where[warp] = (warp * C::kStages + stage) * C::kStage;
    __syncthreads();
    const bool whole = seg.t0 == 0 && seg.t1 == seg.n;
    const int slot = 2 * blockIdx.x + (seg.t0 > 0 ? 0 : 1);
    float* cl_out = reinterpret_cast<float*>(smem + C::kOffQ);
    for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      float2 w[kWarps];
      float top = kNegInf, sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        w[j] = ml[j * 16 + r];
        top = fmaxf(top, w[j].x);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float f = part_weight(w[j], top);
        if (f == 0.0f && w[j].y == w[j].y) continue;  // without a tile its stage is as it was
        sum += w[j].y * f;
        const float4 v = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(smem + where[j]) + r * D + ((d4 ^ (r & 7)) << 2));
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (p.cluster) {
        *reinterpret_cast<float4*>(cl_out + r * D + 4 * d4) = acc;
        if (d4 == 0) reinterpret_cast<float2*>(smem + C::kOffPart)[r] = make_float2(top, sum);
      } else if (whole) {
        const float inv = inverse(sum);
        const int64_t row = (int64_t)seg.b * a.Hq + h0 + r0 + r;
        store_out4<T>(a.out, row * D + 4 * d4,
                      sum == sum ? make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv)
                                 : make_float4(sum, sum, sum, sum));
        if (a.lse && d4 == 0) a.lse[row] = top * kLn2 + logf(sum);
      } else {
        const int64_t row = (int64_t)slot * C::kHeads + r;
        *reinterpret_cast<float4*>(p.part + row * D + 4 * d4) = acc;
        if (d4 == 0) p.ml[row] = make_float2(top, sum);
      }
    }
    __syncthreads();
    // a (sequence, row block) that begins here and goes on in the next CTAs
    if (tid == 0 && seg.t0 == 0 && seg.t1 < seg.n && !p.cluster)
      p.note[blockIdx.x] = Note{seg.b, seg.vh, (int)((seg.u + units(seg.n) - 1) / per), 0};
    next_segment<kT>(seg, p, u1);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (p.cluster == 0) return;

  // ---- the cluster's parts, joined in order by all its CTAs ------------------------------
  const int id = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster, vh = id % p.VH;
  float2* part_ml = reinterpret_cast<float2*>(smem + C::kOffPart);
  if (mine_tiles == 0 && tid < 16) part_ml[tid] = make_float2(kNegInf, 0.0f);
  cluster_sync();
  const int r0 = (vh % p.HC) * C::kHeads, rows = min(p.G - r0, C::kHeads);
  for (int i = rank * kWarps * 32 + tid; i < rows * (D / 4); i += p.cluster * kWarps * 32) {
    const int r = i / (D / 4), d4 = i % (D / 4);
    float2 w[kCluster];
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kCluster; ++j)
      if (j < p.cluster) {
        w[j] = peer_ld2(peer(smem_at(part_ml + r), j));
        top = fmaxf(top, w[j].x);
      }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kCluster; ++j)
      if (j < p.cluster && !(w[j].y == 0.0f)) {  // (a CTA without a tile has no sums)
        const float f = part_weight(w[j], top);
        const float4 v = peer_ld4(peer(smem_at(smem + C::kOffQ) + 4 * (r * D + 4 * d4), j));
        sum = fmaf(w[j].y, f, sum);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
    const float inv = inverse(sum);
    const int64_t row = (int64_t)(id / p.VH) * a.Hq + (vh / p.HC) * p.G + r0 + r;
    store_out4<T>(a.out, row * D + 4 * d4,
                  sum == sum ? make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv)
                             : make_float4(sum, sum, sum, sum));
    if (a.lse && d4 == 0) a.lse[row] = top * kLn2 + logf(sum);
  }
  cluster_sync();  // a CTA's shared memory stays until all have read it
}

// Joins the parts of a (sequence, row block) that begins in CTA blockIdx.x of
// the first kernel and goes on in the CTAs after it; blockIdx.y is the row.
// Threads: column quarters by groups of parts, summed in a fixed order.
template <Act T, int D, int kHeads>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(Args p) {
  constexpr int kCols = D / 4, kGroups = 256 / kCols;
  __shared__ float tops[8], sums[kGroups];
  __shared__ float4 acc_s[kGroups][kCols];
  pdl_release();
  pdl_wait();
  const Note note = p.note[blockIdx.x];
  if (note.b < 0) return;
  const int r = blockIdx.y, r0 = (note.vh % p.HC) * kHeads;
  if (r0 + r >= p.G) return;
  const int parts = note.last - (int)blockIdx.x + 1, tid = threadIdx.x;
  auto row_of = [&](int i) {
    return (int64_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * kHeads + r;
  };
  float top = kNegInf;
  for (int i = tid; i < parts; i += 256) top = fmaxf(top, p.ml[row_of(i)].x);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, i));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
  const int grp = tid / kCols, d4 = tid % kCols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.0f;
#pragma unroll 4
  for (int i = grp; i < parts; i += kGroups) {
    const int64_t row = row_of(i);
    const float2 w = p.ml[row];
    const float4 v = *reinterpret_cast<const float4*>(p.part + row * D + 4 * d4);
    const float f = part_weight(w, top);
    sum = fmaf(w.y, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  acc_s[grp][d4] = acc;
  if (d4 == 0) sums[grp] = sum;
  __syncthreads();
  if (grp != 0) return;
  for (int i = 1; i < kGroups; ++i) {
    const float4 v = acc_s[i][d4];
    sum += sums[i];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float inv = inverse(sum);
  const int64_t row = (int64_t)note.b * p.a.Hq + (note.vh / p.HC) * p.G + r0 + r;
  store_out4<T>(p.a.out, row * D + 4 * d4,
                sum == sum ? make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv)
                           : make_float4(sum, sum, sum, sum));
  if (p.a.lse && d4 == 0) p.a.lse[row] = top * kLn2 + logf(sum);
}

// How many clusters of the kernel the current device runs at once (0: not
// known; asked once a device).
template <Act T, int D, bool kI8, int kBlocks>
int resident_clusters() {
  using C = Cfg<T, D, kI8, kBlocks>;
  static std::atomic<int> known[64];  // one more than the answer
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_decode_kernel<T, D, kI8, kBlocks>, &cfg) != cudaSuccess) {
      static_cast<void>(cudaGetLastError());
      n = 0;
    }
    known[dev].store(++n, std::memory_order_relaxed);
  }
  return n - 1;
}

template <Act T, int D, bool kI8, int kBlocks>
cudaError_t launch(const DecodeArgs& a, void* ws, cudaStream_t st) {
  using C = Cfg<T, D, kI8, kBlocks>;
  constexpr int kCtas = kSms * C::kPerSm;
  static_assert(kCtas <= kMaxCtas, "the workspace has room for every CTA's parts");
  Args p;
  p.a = a;
  p.G = (int)(a.Hq / a.c.kv_heads);
  p.HC = (p.G + C::kHeads - 1) / C::kHeads;
  p.VH = (int)a.c.kv_heads * p.HC;
  p.whole = a.c.page_tokens % C::kT == 0;
  p.part = static_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(p.part + (size_t)2 * kCtas * C::kHeads * D);
  p.note = reinterpret_cast<Note*>(p.ml + (size_t)2 * kCtas * C::kHeads);
  auto kern = attn_decode_kernel<T, D, kI8, kBlocks>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // Few short sequences: a cluster a (sequence, row block), whose CTAs join their
  // parts themselves (one launch).  Up to two tiles a warp: one sequence of 8 x 5
  // heads of 128, fp32 over bf16, takes 6.1 us for 6.9 at 1 token, 8.4 for 9.3 at
  // 1000, but 11.1 for 10.2 at 2000; 4 x 7 heads of 64 in bf16 5.3 for 8.4 and 6.6
  // for 9.5.  And while all run at once: 56 clusters, which do not, took 14.1 for
  // 10.0.
  p.cluster = a.table_width * a.c.page_tokens <= 2 * kCluster * kWarps * C::kT &&
                      a.B * p.VH <= resident_clusters<T, D, kI8, kBlocks>()
                  ? kCluster
                  : 0;
  if (p.cluster)
    return launch_pdl_cluster(kern, dim3((unsigned)(a.B * p.VH * p.cluster)), (unsigned)p.cluster,
                              dim3(kWarps * 32), C::kSmem, st, p);
  e = launch_pdl(kern, dim3(kCtas), dim3(kWarps * 32), C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  const int rows = p.G < C::kHeads ? p.G : C::kHeads;
  return launch_pdl(attn_decode_join_kernel<T, D, C::kHeads>, dim3(kCtas, (unsigned)rows), dim3(256),
                    0, st, p);
}

template <Act T, bool kI8>
cudaError_t by_dim(const DecodeArgs& a, void* ws, cudaStream_t st) {
  const bool two = a.Hq / a.c.kv_heads > 8;
  switch (a.c.head_dim) {
    case 64: return two ? launch<T, 64, kI8, 2>(a, ws, st) : launch<T, 64, kI8, 1>(a, ws, st);
    case 128: return two ? launch<T, 128, kI8, 2>(a, ws, st) : launch<T, 128, kI8, 1>(a, ws, st);
    default: return launch<T, 256, kI8, 1>(a, ws, st);  // two blocks' output would not fit the registers
  }
}

}  // namespace

size_t attn_decode_workspace(int64_t, int64_t, int64_t, int64_t D) {
  return (size_t)kMaxCtas * (2 * 16 * ((size_t)D * 4 + 8) + sizeof(Note));
}

cudaError_t launch_attn_decode(const DecodeArgs& a, void* ws, cudaStream_t st) {
  const bool i8 = a.c.type == PTQ_KV_I8;
  if (a.t == Act::F32)
    return i8 ? by_dim<Act::F32, true>(a, ws, st) : by_dim<Act::F32, false>(a, ws, st);
  return i8 ? by_dim<Act::BF16, true>(a, ws, st) : by_dim<Act::BF16, false>(a, ws, st);
}

}  // namespace ptq
