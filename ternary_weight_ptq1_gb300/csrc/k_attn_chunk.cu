// k_attn_chunk.cu -- attention of chunks of new tokens over their paged
// key-value cache, all of it or a sliding window and the first tokens, on the
// 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - m),  O = P V,  out = O / sum P
//
// over the tokens j <= p of a query's position p, with a window those with
// p - window < j or j < sinks.  4 head_dim operations a visible (query, key) pair and
// query head against one exponential: on chunks of prompts the chain of an S, its
// softmax and its product bounds it (the tensor cores are busy 62% of the time), on a
// few tokens each over long contexts the bytes of the cache over bf16; over int8 the
// warps that spread codes, one unit's waits, reads, 130 instructions and stores after
// another.
//
// Measured in CUDA graphs, causal: chunks of 1300 to 2048 tokens of three prompts over
// up to 14,000 before them, 8 x 5 heads of 128, bf16 in 582 us (1340 TFLOP/s; with
// nothing waited for between calls 624, under the power limit); 8192 tokens over
// themselves in 520 (1320), through int8 in 817 (840), 4 x 6 of 256 in 704 (1170) and
// 1229 (670), 4 x 7 of 64 in 332 (725) and 530 (455); 64 sequences' 1 to 5 new tokens over
// up to 8192, 8 x 8 of 128, over bf16 in 167 us (5.7 TB/s, 84% of the copy rate), over
// int8 in 205 (2.4); 12 chunks of up to 900 under a window of 1024 + 4, 4 x 6 of 256,
// int8 in 188; 4 tokens over 781 in 14.4.  Reading the rows back and the kernel of whole
// prompts take 463 us for the first of those 8192, over int8 or bf16, 542 and 262 for the others.
//
// Keys.  The tokens that some query of a Q tile sees are counted through: the
// first `sinks`, then those of the window, so first tokens share a tile of 128
// keys with others and hidden ones cost nothing.  Four warps copy a tile's rows out of
// the pages (cp.async, a lane finds the page of a row): any page size packs full
// tiles, and rows that are not there are zeros.  (With zeros for every row, nothing read
// from the pages, 8192 tokens take 510 us for 527, 4 x 7 of 64 326 for 332: what the
// tensor memory accelerator, which wants whole pieces of pages, could save is within
// that.)  Over int8 eight warps each copy codes to a place of their own and spread them
// to bf16 for the products (times 2^-16), which is exact (four take 286 us for 266 on the
// 64 sequences); a score is then multiplied by its key's scale and a probability by its
// value's, in fp32, before P is rounded to bf16.
//
// Tile.  128 rows of Q are tpt tokens of hg query heads that share a kv head.  S, P
// and O live in TMEM as in the kernel of whole prompts: P goes back over S as bf16
// and is the A operand of the second product (both operands have one type, and two
// terms of P would add half to its work: 2^-9 of each weight, which takes an output's
// error from its own rounding's 1.7e-3 to 2.3e-3); the maximum that it refers to moves
// when a row's grows by more than 2^8.  A CTA works on two S at a time (head_dim up
// to 128): of two Q tiles, neighbours in the sequence, that share each K and V
// tile; or, where a sequence's queries fill one, of the one tile over every other
// tile of keys, with an O each that are added at the end.  At head_dim 256 the
// one tile's S has two buffers.
//
// Work.  Runs of queries (the CTA's Q tiles) times head blocks, in order, cost
// their keys and a start of kLead; each CTA gets an equal stretch of that order,
// cut at tiles of keys: one long context spreads over all SMs, ragged batches end
// together.  The lengths are on the device: every CTA adds them up (in closed form
// for a sequence) and one of its warps walks its stretch.  A run that is cut
// leaves its sums, relative to their maxima, in the workspace, and a second kernel
// joins them in order; a CTA joins those of its own part every 2^15 keys.  (A start of
// 128 keys: 64 sequences over int8 231 us, of 256 204, of 512 202, of 1024 217; three
// chunks 613, 597, 590, 601.)
//
// What runs between two products is kept short: an issuing warp that works out its places
// after its waits, or votes on each wait, takes 610 us for 518 at 8192 tokens.
//
// A key that a row does not see has P = 0, and 0 times a non-finite value is NaN.
// Over int8 a row is not finite by its scale: such scales enter as 0, and rows that
// see one are made NaN.  Over bf16 rows whose sum is finite and whose output is not
// are looked at, and computed again where no value that they see explains a dimension
// of it.
//
// Every wait is bounded, to some 6 s in which no warp computes rows again; one that
// runs out raises the device status word and the CTA drains what it has in flight and
// exits.
#include <cuda_bf16.h>

#include <type_traits>

#include "attn_row.cuh"
#include "attn_tc.cuh"
#include "ptq_internal.cuh"

namespace ptq {
namespace {

constexpr int kCtas = (int)kSms;
constexpr int kLead = 512;   // cost of a run's start, in keys
constexpr int kLeast = 256;  // the shortest stretch of a CTA
constexpr int kScales = 8;   // tiles whose scales are in shared memory
constexpr float kCodeUp = 0x1p16f, kCodeDown = 0x1p-16f;  // codes enter the products as 2^-16 of themselves
constexpr int kItems = 4;    // items on their way from the warp that plans to the others
// A sum of n terms made one after the other is off by up to n / 2 units of 2^-23 where it truncates
// (as the tensor core does, 16 keys a term: 2^20 keys of one score were off by 1.5%), n / 2 half ones
// where it rounds.  So O and the row's four sums go over kPiece tiles of keys, 2^15, off by
// 2^-13 and 2^-12 at most, and are then joined.  (A row's sums joined every 16 tiles beside: 8192 tokens
// of 4 x 6 of 256 715 us for 703.)
constexpr int kPiece = 256;

template <int D, bool kI8>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;    // Q tiles of a CTA
  // A K or V tile passes through the ring in one unit, or two: K by columns,
  // V by keys, as the products use them up.
  static constexpr int kUnits = D == 256 ? 2 : 1;
  static constexpr int kCols = D / kUnits;           // columns of a K unit
  static constexpr int kVKeys = kKeys / kUnits;      // keys of a V unit
  static constexpr int kUnit = kKeys * kCols * 2;    // bytes
  static constexpr int kRing = kI8 ? (D == 64 ? 6 : 3) : (D == 64 ? 8 : 5);
  // Units on their way at most (int8: the places that they land in).
  static constexpr int kAhead = kI8 ? (D == 64 ? 6 : 2) : D == 128 ? 2 : 3;
  static constexpr int kStage = kI8 ? kUnit / 2 : 0;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSoftmax = 4 * kTiles;        // softmax warps
  static constexpr int kFeeds = kI8 ? 8 : 4;          // warps that feed
  static constexpr int kThreads = 32 * (kSoftmax + kFeeds + 4);
  // Registers a thread.  Two Q tiles, bf16: 512 threads get 128 each at launch (65,536
  // in all); 256 softmax threads take 168, 128 that feed keep 96 and 128 others
  // 80 (65,536); int8: 640 get 96 (61,440), 256 take 152, 256 keep 56 and 128 keep 64
  // (61,440).  One, bf16: 384 get 168 (64,512); 128 take 232, 128 keep 128, 128 keep
  // 104 (59,392); int8: 512 get 128 (65,536), 128 take 232, 256 keep 80, 128 keep 104 (63,488).
  static constexpr int kRegsSoftmax = kTiles == 1 ? 232 : kI8 ? 152 : 168;
  static constexpr int kRegsFeed = kTiles == 1 ? (kI8 ? 80 : 128) : kI8 ? 56 : 96;
  static constexpr int kRegsOther = kTiles == 1 ? 104 : kI8 ? 64 : 80;
  static constexpr int kOffRing = kTiles * kQ;
  static constexpr int kOffStage = kOffRing + kRing * kUnit;
  // int8: K and V scales of each tile, and a bit for each V scale that is not finite;
  // and scales of 1
  static constexpr int kOffScale = kOffStage + kAhead * kStage;
  static constexpr int kOffOdd = kOffScale + (kI8 ? kScales * 2 * kKeys * 4 : 0);
  static constexpr int kOffOnes = kOffOdd + (kI8 ? kScales * 16 : 0);
  static constexpr int kOffBar = kOffOnes + (kI8 ? kKeys * 4 : 0);
  // full[kRing] empty[kRing] q[2] q free[2] s[2] p[2][2] o[2] o free[2] pv[2] turn[2]
  // item full[kItems] item empty[kItems] sums full, empty, scales[kScales], done
  static constexpr int kBars = 2 * kRing + 4 + 2 + 4 + 2 + 2 + 2 + 2 + 2 * kItems + 2 + kScales + 1;
  static constexpr int kOffItem = (kOffBar + 8 * kBars + 15) / 16 * 16;
  static constexpr int kOffSums = kOffItem + kItems * 64;  // (maximum, sum) of the second half's rows
  static constexpr int kOffBad = kOffSums + (kTiles == 2 ? kRows * 8 : 0);
  static constexpr int kOffMisc = kOffBad + kFeeds * 16 * 4;
  static constexpr int kSmem = kOffMisc + 16;
};
static_assert(Cfg<128, false>::kSmem <= 227 * 1024 && Cfg<256, false>::kSmem <= 227 * 1024 &&
                  Cfg<128, true>::kSmem <= 227 * 1024 && Cfg<256, true>::kSmem <= 227 * 1024, "shared memory");
// The scales of a tile stay until its P is written: its V is released after that.  When the
// copies of K tile j are issued the units before the last kRing + kAhead are released: all up to
// V tile j - kScales at least.
static_assert(2 * (kScales - 1) >= Cfg<64, true>::kRing + Cfg<64, true>::kAhead + 1 &&
                  4 * (kScales - 2) >= Cfg<256, true>::kRing + Cfg<256, true>::kAhead + 1, "scales");
static_assert(Cfg<64, true>::kAhead <= 15 && Cfg<64, false>::kAhead <= 15, "kinds of 16 units");

// A run that is cut: what the second kernel joins.
struct Note {
  int64_t row;  // first query and head of the run, among Tq Hq rows
  int tokens;   // 0: none
  int slot;     // of its first part, in its CTA; the others' is 0
  int last;     // CTA of its last part
  int pad[3];
};

struct Args {
  ChunkArgs a;
  int G, hg, tpt;  // query heads of a kv head; heads and tokens of a Q tile
  int heads;       // head blocks in all
  int run;         // queries of an item: the Q tiles' tokens
  int part_rows;   // rows of a part
  Divider by_G, by_hg, by_run, by_page;
  // A score in units of log2 is S times scale2 (over int8 also its key's scale, times key_up: 2^16 is in
  // the one or, for a softmax_scale that leaves no room for it, in the other).
  float scale2, key_up;
  float* part;     // [CTA][2][part_rows][D] output sums
  float2* ml;      // [CTA][2][part_rows], the maximum and sum they refer to
  Note* note;      // [CTA]
};

// A CTA's next piece of work: the Q tiles of one run and head block, over tiles
// of the keys that the run sees, kPiece at most (the next piece goes on from its sums).  b < 0: no more.
struct Item {
  int b, q0, nq, first;  // the sequence, its first query's row, its queries, the run's first
  int h, hq0;            // kv head, first query head
  int nk;                // cached tokens of the sequence
  int skip, nv;          // tokens hidden after the first `sinks`; tokens that the run sees
  int t0, tiles;         // this part's tiles
  int n[2];              // tiles of each Q tile, or (split) of each half
  int split;             // one Q tile, its key tiles dealt out to both S
  int slot;              // part of the workspace and kWhole, kOnto; -1: the whole run at once
  int r0;                // the run's first tile in this CTA
};
// The item ends its run, all of which is this CTA's; the part has the sums of tiles [r0, t0).
constexpr int kWhole = 2, kOnto = 4;
static_assert(sizeof(Item) <= 64, "its place in shared memory");

// ---- the order of the work -----------------------------------------------------------

struct Seq {
  int q0, nq, nk;
};
__device__ __forceinline__ Seq seq_of(const ChunkArgs& a, int b) {
  const int Tq = (int)a.Tq;
  const int64_t most = a.table_width * a.c.page_tokens;
  const int n = __ldg(a.lens + b);
  const int q0 = clamped(__ldg(a.cu_q + b), Tq), q1 = clamped(__ldg(a.cu_q + b + 1), Tq);
  return {q0, max(0, q1 - q0), n < 0 ? 0 : n > most ? (int)most : n};
}

// The sum of max(0, at + i step) for i < n, where step n < 2^31.
__device__ __forceinline__ int64_t ramp(const Args& p, int64_t at, int n) {
  if (n <= 0 || at + (int64_t)p.run * (n - 1) <= 0) return 0;
  const int i0 = at > 0 ? 0 : p.by_run((int)-at) + 1;
  const int64_t k = n - i0, first = at + (int64_t)i0 * p.run;
  return k * first + p.run * (k * (k - 1) / 2);
}

__device__ __forceinline__ int runs_of(const Args& p, int nq) { return p.by_run(nq + p.run - 1); }

// The cost of the first r runs of a sequence.
__device__ __noinline__ int64_t cost_of(const Args& p, const Seq& s, int r) {
  const int64_t base = (int64_t)s.nk - s.nq;
  int64_t sum = (int64_t)kLead * r + ramp(p, base + p.run, r);
  if (r > 0 && (int64_t)r * p.run > s.nq) sum -= (int64_t)r * p.run - s.nq;  // the last run is shorter
  if (p.a.window) sum -= ramp(p, base + 1 - p.a.window - p.a.sinks, r);
  return sum;
}

// Tokens that run r sees, and those hidden after the first ones.
__device__ __forceinline__ int tokens_of(const Args& p, const Seq& s, int r, int* skip) {
  const int end = max(0, s.nk - s.nq + min((r + 1) * p.run, s.nq));
  const int from = max(0, s.nk - s.nq + r * p.run + 1);
  *skip = p.a.window ? max(0, max(0, from - p.a.window) - p.a.sinks) : 0;
  return end - *skip;
}

__device__ __forceinline__ int tiles_of(int tokens) { return (int)(((unsigned)tokens + kKeys - 1) / kKeys); }

// The first tile of a run (of n, which begins at unit `start`) that is not before unit u.
__device__ __forceinline__ int tile_at(int64_t u, int64_t start, int n) {
  const int64_t k = u - start - kLead;
  return k <= 0 ? 0 : (int)min((int64_t)n, (k + kKeys - 1) / kKeys);
}

// ---- rows again ------------------------------------------------------------------------

// Eight consecutive values of a cached row, in fp32 (int8: codes).
template <bool kI8>
__device__ __forceinline__ void row8(const void* p, int64_t e, float (&x)[8]) {
  if constexpr (kI8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + e));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
  } else {
    load_bf16(static_cast<const uint16_t*>(p) + e, x);
  }
}

// A lane's D / 32 columns of a cached row.
template <int D, bool kI8>
__device__ __forceinline__ void columns(const void* p, int64_t row, int lane, float (&x)[D / 32]) {
  constexpr int N = D / 32;
  if constexpr (kI8) {
    const int8_t* q = static_cast<const int8_t*>(p) + row * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)__ldg(q + i);
  } else {
    load_bf16(static_cast<const uint16_t*>(p) + row * D + lane * N, x);
  }
}

// What a row sees of its run's tokens v: v < end and (v >= from or v < sinks).
struct Sight {
  int end, from, sinks;
  __device__ __forceinline__ bool sees(int v) const { return v < end && (v >= from || v < sinks); }
};

// The row of the cache of the run's token v; -1: its page is none.
__device__ __forceinline__ int64_t cached_row(const ChunkArgs& a, const Item& it, int v) {
  const unsigned ps = (unsigned)a.c.page_tokens, j = (unsigned)v + (v >= a.sinks ? it.skip : 0);
  const int page = __ldg(a.table + it.b * a.table_width + j / ps);
  if ((unsigned)page >= (unsigned)a.c.pages) return -1;
  return ((int64_t)page * a.c.kv_heads + it.h) * ps + j % ps;
}

// One query row by a warp over the run's tokens [v0, v1): 32 keys at a time, a
// lane's own key for the scores and its own columns for the output.  Where the
// weights' sum is large the sums of values near the largest overflow although
// their mean does not: then again with weights 2^-40 times as large.  Sums go over kRowKeys
// keys and are then joined.
constexpr int kRowKeys = 4096;
template <int D, bool kI8>
__device__ __noinline__ void attend_row(const Args& p, const Item& it, int64_t row, Sight sight, int v0, int v1,
                                        float* part, float2* ml) {
  constexpr int N = D / 32;
  const ChunkArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t t = row / a.Hq;
  const uint16_t* q = a.q + t * a.q_stride + (row - t * a.Hq) * D;
  const int stop = min(v1, sight.end);
  RowState<D> all;
  float small = 1.0f;
#pragma unroll 1
  for (;;) {
    all = RowState<D>();
    RowState<D> s;
#pragma unroll 1
    for (int v = v0; v < stop; v += 32) {
      const int mine = v + lane;
      const bool in = mine < stop && sight.sees(mine);
      const int64_t at = in ? cached_row(a, it, mine) : -1;
      float x = in ? __int_as_float(0x7fc00000) : kNegInf, vs = 1.0f;
      if (at >= 0) {
        x = 0.0f;
#pragma unroll 8
        for (int d = 0; d < D; d += 8) {
          float k[8], y[8];
          row8<kI8>(a.c.k, at * D + d, k);
          row8<false>(q, d, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) x = fmaf(k[i], kI8 ? y[i] * kCodeDown : y[i], x);
        }
        if constexpr (kI8) x *= __ldg(a.c.k_scale + at) * p.key_up, vs = __ldg(a.c.v_scale + at);
        x *= p.scale2;
      }
      const float w = s.weigh(x) * (small * vs);
      const unsigned there = __ballot_sync(~0u, at >= 0);
      constexpr int kBatch = D == 256 ? 4 : 8;  // values loaded together
#pragma unroll 1
      for (int e0 = 0; e0 < 32; e0 += kBatch) {
        float y[kBatch][N];
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
          columns<D, kI8>(a.c.v, max(__shfl_sync(~0u, at, e0 + e), (int64_t)0), lane, y[e]);
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const float we = __shfl_sync(~0u, w, e0 + e);
          if (there >> (e0 + e) & 1) {  // (0 times a hidden value may be NaN)
#pragma unroll
            for (int i = 0; i < N; ++i) s.o[i] = fmaf(we, y[e][i], s.o[i]);
          }
        }
      }
      if ((v - v0) % kRowKeys == kRowKeys - 32 || stop - v <= 32) {
        float l = s.l;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(~0u, l, i);
        all.join(s.m, l, s.o);
        s = RowState<D>();
      }
    }
    bool fine = true;
#pragma unroll
    for (int i = 0; i < N; ++i) fine = fine && fabsf(all.o[i]) < -kNegInf;
    if (small != 1.0f || !(all.l == all.l) || __all_sync(~0u, fine)) break;
    small = 0x1p-40f;
  }
  if (part) {
    if (lane == 0) *ml = make_float2(small == 1.0f ? all.m : all.m + 40.0f, all.l * small);
#pragma unroll
    for (int i = 0; i < N; ++i) part[lane * N + i] = all.o[i];
  } else {
    const float inv = all.l == 0.0f ? 0.0f : 1.0f / (all.l * small);
#pragma unroll
    for (int i = 0; i < N; ++i)
      a.out[row * D + lane * N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(all.o[i] * inv));
  }
}

// The rows `again` of a warp (a lane a row) whose sum is finite and whose output is not.  A
// value that a row sees and that is not finite leaves its column so, rightly.  The row is
// computed again where a column of its output is not finite and has none of those: a hidden
// one (0 times it is NaN) did it, or the sum of large values overflowed (P may be 2^8 times a
// probability).  The tokens of [v0, v1) that all of the rows see are looked at together, until
// they explain every column.  8192 tokens, 8 x 5 heads of 128, 0.56 ms: with the first token's value
// infinite, which all rows see, 0.75 (21 when each row was looked at alone), with the middle one's 26
// (426), with the last one's 37 (184).
template <int D>
__device__ __noinline__ unsigned spoilt(const Args& p, const Item& it, unsigned again, int64_t row, const float* part,
                                        Sight sight, int v0, int v1) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const bool mine = again >> lane & 1;
  // this lane's columns (a bit each) of row `who` as it was written that are not finite
  auto bad_of = [&](int who) {
    const int64_t r = __shfl_sync(~0u, row, who);
    const volatile float* from =
        reinterpret_cast<const float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(part), who));
    const volatile uint16_t* out = p.a.out + r * D + lane * N;
    unsigned bad = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = from ? from[lane * N + i] : __uint_as_float((uint32_t)out[i] << 16);
      if (!(fabsf(y) < -kNegInf)) bad |= 1u << i;
    }
    return bad;
  };
  auto look = [&](int v, unsigned& found) {  // this lane's columns of token v
    const int64_t at = cached_row(p.a, it, v);
    float y[N];
    if (at >= 0) {
      columns<D, false>(p.a.c.v, at, lane, y);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(fabsf(y[i]) < -kNegInf)) found |= 1u << i;
    }
  };
  unsigned all = 0, known = 0;
#pragma unroll 1
  for (unsigned rest = again; rest; rest &= rest - 1) all |= bad_of(__ffs(rest) - 1);
  // tokens that all of the rows see, [sinks, from) left out
  const int end = min(v1, __reduce_min_sync(~0u, mine ? sight.end : v1)),
            from = __reduce_max_sync(~0u, mine ? sight.from : 0), sinks = sight.sinks;
  const int gap0 = max(v0, min(sinks, end)), gap1 = min(from, end);
#pragma unroll 1
  for (int v = v0; v < end; v += 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (v + e < end && !(v + e >= gap0 && v + e < gap1)) look(v + e, known);
    if (!__any_sync(~0u, all & ~known)) return 0u;
  }
  unsigned todo = 0;
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int who = __ffs(again) - 1;
    const unsigned bad = bad_of(who) & ~known;
    if (!__any_sync(~0u, bad)) continue;
    const Sight s{__shfl_sync(~0u, sight.end, who), __shfl_sync(~0u, sight.from, who), sinks};
    unsigned seen = 0;  // by this row among the others
#pragma unroll 4
    for (int v = gap0; v < gap1; ++v)
      if (s.sees(v)) look(v, seen);
#pragma unroll 4
    for (int v = max(v0, end); v < v1; ++v)
      if (s.sees(v)) look(v, seen);
    if (__any_sync(~0u, bad & ~seen)) todo |= 1u << who;
  }
  return todo;
}

template <int D, bool kI8>
__device__ __noinline__ void repair(const Args& p, const Item& it, unsigned again, int64_t row, Sight sight, int v0,
                                    int v1, float* part, float2* ml, volatile int* state) {
  const Busy busy(state);
  if constexpr (!kI8) again = spoilt<D>(p, it, again, row, part, sight, v0, v1);
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int who = __ffs(again) - 1;
    const Sight s{__shfl_sync(~0u, sight.end, who), __shfl_sync(~0u, sight.from, who), sight.sinks};
    const int64_t r = __shfl_sync(~0u, row, who);
    float* to = reinterpret_cast<float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(part), who));
    float2* mt = reinterpret_cast<float2*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(ml), who));
    attend_row<D, kI8>(p, it, r, s, v0, v1, to, mt);
  }
}

// ---- copies ------------------------------------------------------------------------------

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
template <int N>
__device__ __forceinline__ void copies_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// All groups of copies but the last n (or fewer) have landed.
__device__ __forceinline__ void copies_but(int n) {
  switch (n) {
    case 0: return copies_but<0>();
    case 1: return copies_but<1>();
    case 2: return copies_but<2>();
    case 3: return copies_but<3>();
    default: return copies_but<4>();
  }
}

// Two of the four int8 codes of x as bf16, times 2^-16: under the exponent of 2^-9 a byte's low
// seven bits are 2^-9 + them and its top bit is 2^-9 or 2^-8, and their difference is the code.
// q times such codes, added up over 256 columns, stays under 2^127 for any bf16 q (times whole codes it
// passed 2^128 from q of 2^113 on), and is exact down to the smallest q, 2^-133: fp32 holds 2^-149.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes(uint32_t x) {
  const uint32_t w = __byte_perm(x, 0x3b3b3b3bu, kSel), a = w & 0xff7fff7fu, b = w & 0xff80ff80u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// The weight of sums with maximum m and sum l among sums of maximum top.
// l = 0: no key.  m = -inf with l != 0: NaN scores.
__device__ __forceinline__ float weight(float m, float l, float top) {
  return l == 0.0f ? 0.0f : m == kNegInf ? 1.0f : exp2_fast(m - top);
}

__device__ __forceinline__ void shared4(uint32_t at, float (&x)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at));
}

__device__ __forceinline__ uint32_t low_bits(int n) {  // n below 0: none, above 32: all
  return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
}

// A row's output, w0 O0 + w1 O1, from TMEM, as bf16 or (a part) fp32; whether it is finite.
// how: 1 both O, 2 the row is one, 4 a part, 8 NaN, 16 O0 has a key's product (else it may be
// anything), 32 O1 has one.  (A weight says neither: it is 0 also where an O's scores are far
// below the other's, and 0 times a value that is not finite is NaN.)  (Called: inlined its registers are kept from the scores', which then spill.)
template <int D, bool kOnto>
__device__ __forceinline__ bool put_columns(uint32_t o0, uint32_t o1, float w0, float w1, char* to, unsigned how,
                                            const float* before, float wb) {
  uint64_t checked = pair(0.0f, 0.0f);
  const uint64_t ww0 = pair(w0, w0), ww1 = pair(w1, w1), zero2 = pair(0.0f, 0.0f);
  __syncwarp();
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16], x[16] = {};
    tmem_ld16(o0 + c, o);
    if (__any_sync(~0u, how & 1)) tmem_ld16(o1 + c, x);  // (of the whole warp)
    tmem_wait_ld();
    if (!(how & 16)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = 0u;
    }
    if (!(how & 32)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0u;
    }
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      uint64_t y = mul2(pair(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), ww0);
      y = fma2(pair(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), ww1, y);
      if constexpr (kOnto) {
        if (how & 2) y = fma2(pair(before[c + e], before[c + e + 1]), pair(wb, wb), y);
      }
      checked = fma2(y, zero2, checked);  // 0 as long as every value is finite
      float y0, y1;
      unpair(y, y0, y1);
      if (how & 8) y0 = y1 = __int_as_float(0x7fc00000);
      o[e] = __float_as_uint(y0), o[e + 1] = __float_as_uint(y1);
    }
    if (how & 2) {
      if (how & 4) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint4*>(to + 4 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(to + 16) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    to += how & 4 ? 64 : 32;
    __syncwarp();
  }
  float lo, hi;
  unpair(checked, lo, hi);
  return lo + hi == 0.0f;
}
template <int D>
__device__ __noinline__ bool put_row(uint32_t o0, uint32_t o1, float w0, float w1, char* to, unsigned how) {
  return put_columns<D, false>(o0, o1, w0, w1, to, how, nullptr, 0.0f);
}

// The output of a piece whose run has pieces before it in this CTA: w0 O0 + w1 O1, of maximum m and
// sum l, joined with the part's sums; back into the part, or the row's output.  Bits: 1 all is finite,
// 2 the row is NaN by a value's scale, 4 its sum is no NaN.
template <int D, bool kI8>
__device__ __noinline__ unsigned put_row_onto(const Args& p, uint32_t o0, uint32_t o1, float w0, float w1, float m, float l,
                                              unsigned how, int64_t part_row, int64_t out_row) {
  float* part = p.part + part_row * D;
  float wb = 0.0f;
  if (how & 2) {
    const float2 before = p.ml[part_row];
    const float top = fmaxf(m, before.x), f = weight(m, l, top);
    wb = weight(before.x, before.y, top);
    w0 *= f, w1 *= f;
    l = l * f + before.y * wb;
    if (kI8 && !(part[0] == part[0])) how |= 8;  // (over int8 a row that sees such a scale is NaN)
    if (how & 4) {
      p.ml[part_row] = make_float2(top, l);
    } else {
      const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
      w0 *= inv, w1 *= inv, wb *= inv;
      if (p.a.lse) p.a.lse[out_row] = l == 0.0f ? kNegInf : (top + __log2f(l)) * kLn2;
    }
  }
  char* to = how & 4 ? reinterpret_cast<char*>(part) : reinterpret_cast<char*>(p.a.out + out_row * D);
  const bool fine = put_columns<D, true>(o0, o1, w0, w1, to, how, part, wb);
  return (fine ? 1u : 0u) | (how & 8 ? 2u : 0u) | (l == l ? 4u : 0u);
}

template <int D, bool kI8>
__global__ void __launch_bounds__(Cfg<D, kI8>::kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ Args p, int* status) {
  using C = Cfg<D, kI8>;
  constexpr int kTiles = C::kTiles;
  constexpr bool kAfter = kTiles == 2;  // the next S goes where P was
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  // ring units; of a Q tile: Q there, Q read; of a slot: S written, the first and
  // second half of P written; of a Q tile: O final, O read, a product with V
  // done (not where S's arrival says it), its turn to issue; items there, read; the
  // second half's sums there, read; a tile's scales there
  uint64_t *full = bars, *empty = bars + C::kRing, *q_full = bars + 2 * C::kRing, *q_free = q_full + 2;
  uint64_t *s_full = q_free + 2, *p_full = s_full + 2, *o_full = p_full + 4,
           *o_free = o_full + 2, *pv_done = o_free + 2, *turn = pv_done + 2, *item_full = turn + 2,
           *item_free = item_full + kItems, *ml_full = item_free + kItems, *ml_free = ml_full + 1,
           *scales = ml_free + 1, *all_done = scales + kScales;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* state = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

  const ChunkArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kFeed = C::kSoftmax, kMma = kFeed + C::kFeeds, kPlan = kMma + kTiles, kWarps = C::kThreads / 32;

  pdl_release();
  pdl_wait();

  // ---- this CTA's stretch of the work, [u0, u1), and the sequence that it begins in ------
  int64_t u0, u1, per, seq_start = 0;
  int seq = -1;
  {
    int64_t* scan = reinterpret_cast<int64_t*>(smem);  // (the places of Q, not yet used)
    int64_t mine = 0;
    auto cost = [&](int64_t b) {
      if (b >= a.B) return (int64_t)0;
      const Seq s = seq_of(a, (int)b);
      return cost_of(p, s, runs_of(p, s.nq)) * p.heads;
    };
    for (int64_t b = threadIdx.x; b < a.B; b += C::kThreads) mine += cost(b);
    int64_t incl = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, incl, i);
      if (lane >= i) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    if (threadIdx.x == 0) p.note[blockIdx.x].tokens = 0;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    per = (total + gridDim.x - 1) / gridDim.x;
    per = max((int64_t)kLeast, (per + kKeys - 1) / kKeys * kKeys);
    u0 = blockIdx.x * per;
    u1 = min(u0 + per, total);
    if (u0 >= total) return;
    int64_t* found = scan + kWarps;  // sequence, its start
    if (a.B <= C::kThreads) {
      const int64_t start = before + incl - mine;
      if (u0 >= start && u0 < start + mine) found[0] = threadIdx.x, found[1] = start;
    } else {
      for (int64_t b0 = 0, base = 0;; b0 += C::kThreads) {
        const int64_t one = cost(b0 + threadIdx.x);
        int64_t upto = one;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const int64_t o = __shfl_up_sync(~0u, upto, i);
          if (lane >= i) upto += o;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        int64_t start = base + upto - one;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) start += scan[w];
          base += scan[w];
        }
        if (u0 >= start && u0 < start + one) found[0] = b0 + threadIdx.x, found[1] = start;
        if (u0 < base) break;
      }
    }
    __syncthreads();
    seq = (int)found[0];
    seq_start = found[1];
    __syncthreads();
  }

  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kFeed && lane == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(full + i, C::kFeeds);
      mbar_init(empty + i, kTiles);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_free + i, kTiles);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + 2 * i, 4);  // the four softmax warps of a tile
      mbar_init(p_full + 2 * i + 1, 4);
      mbar_init(o_full + i, 1);
      mbar_init(o_free + i, 4);
      mbar_init(pv_done + i, 1);
      mbar_init(turn + i, 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_free + i, C::kFeeds + kTiles + C::kSoftmax);  // every warp that reads items
    }
    mbar_init(ml_full, 4);
    mbar_init(ml_free, 4);
    for (int i = 0; i < kScales; ++i) mbar_init(scales + i, C::kFeeds);
    mbar_init(all_done, kTiles);
    *state = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if constexpr (kI8) {
    if (threadIdx.x < kKeys) reinterpret_cast<float*>(smem + C::kOffOnes)[threadIdx.x] = 1.0f;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t ring = smem_addr(smem + C::kOffRing), qs = smem_addr(smem);
  bool ok = true;

  int seen = 0;  // items read
  auto item_ready = [&] { return mbar_test(item_full + seen % kItems, (seen / kItems) & 1); };
  auto item_there = [&] {  // the next one's place
    ok = __all_sync(~0u, bar_wait(item_full + seen % kItems, (seen / kItems) & 1, state));
    return reinterpret_cast<const volatile Item*>(smem + C::kOffItem + seen % kItems * 64);
  };
  auto item_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(item_free + seen % kItems);
    ++seen;
  };
  auto read_item = [&](Item& it) {
    const volatile int* from = reinterpret_cast<const volatile int*>(item_there());
    if (!ok) return false;
    int* to = reinterpret_cast<int*>(&it);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) to[i] = from[i];
    item_done();
    return it.b >= 0;
  };
  if (warp >= kMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
  if (warp == kPlan) {
    // ---- the items of this CTA, one ahead of their use, and their Q tiles -----------------
    int qn[kTiles] = {};  // Q tiles loaded
    Seq s = seq_of(a, seq);
    int64_t each = cost_of(p, s, runs_of(p, s.nq));
    int hb = (int)((u0 - seq_start) / each), r = 0;
    int64_t start = seq_start + hb * each;  // of the run
    {  // the last run that begins at u0 or before
      int lo = 0, hi = runs_of(p, s.nq);
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start + cost_of(p, s, mid) <= u0) lo = mid; else hi = mid;
      }
      r = lo;
      start += cost_of(p, s, r);
    }
    Item it;
    it.b = -1;
    int t1 = 0;    // the end of the run's tiles in this CTA
    int part = 0;  // where its sums go if they are not the whole run's
    while (ok) {
      if (it.b >= 0 && it.t0 + it.tiles < t1) {
        it.t0 += it.tiles;  // the run's next piece
      } else {
        it.b = -1;
        while (start < u1) {
          if (r * (int64_t)p.run >= s.nq) {  // the next head block, or sequence with queries
            r = 0;
            if (++hb == p.heads) {
              hb = 0;
              for (++seq;; seq += 32) {
                const bool some = seq + lane < a.B && seq_of(a, seq + lane).nq > 0;
                const unsigned which = __ballot_sync(~0u, some);
                if (which) {
                  seq += __ffs(which) - 1;
                  break;
                }
                if (seq + 32 >= a.B) break;  // (start is u1 before that)
              }
              s = seq_of(a, min(seq, (int)a.B - 1));
            }
          }
          it.nv = tokens_of(p, s, r, &it.skip);
          const int n = tiles_of(it.nv);
          it.t0 = it.r0 = tile_at(u0, start, n);
          t1 = tile_at(u1, start, n);
          const int64_t begin = start;
          const int this_run = r++;
          start += (int64_t)kLead + it.nv;
          if (it.t0 >= t1 && !(n == 0 && begin >= u0)) continue;
          it.b = seq;
          it.q0 = s.q0, it.nq = s.nq, it.nk = s.nk;
          it.first = this_run * p.run;
          it.hq0 = hb * p.hg;
          it.h = p.by_G(it.hq0);
          it.split = kTiles == 2 && it.first + p.tpt >= it.nq;
          part = begin < u0 ? 0 : 1;
          if (it.t0 == 0 && t1 < n && lane == 0) {
            Note note;
            note.row = (int64_t)(it.q0 + it.first) * a.Hq + it.hq0;
            note.tokens = min(p.run, it.nq - it.first);
            note.slot = part;
            note.last = (int)((begin + kLead + (int64_t)(n - 1) * kKeys) / per);
            p.note[blockIdx.x] = note;
          }
          break;
        }
      }
      if (it.b >= 0) {
        it.tiles = min(t1 - it.t0, kPiece);
        const bool whole = it.r0 == 0 && t1 == tiles_of(it.nv), ends = it.t0 + it.tiles == t1, onto = it.t0 != it.r0;
        it.slot = whole && ends && !onto ? -1 : part | (whole && ends ? kWhole : 0) | (onto ? kOnto : 0);
        if (kTiles == 1) {
          it.n[0] = it.tiles, it.n[1] = 0;
        } else if (it.split) {
          it.n[0] = (it.tiles + 1) / 2, it.n[1] = it.tiles / 2;
        } else {
          const int v = it.nk - it.nq + it.first + p.tpt - it.skip;  // what the first tile's last query sees
          const int n0 = tiles_of(max(v, 0));
          it.n[0] = max(0, min(n0 - it.t0, it.tiles)), it.n[1] = it.tiles;
        }
      }
      if (seen >= kItems)
        ok = __all_sync(~0u, bar_wait(item_free + seen % kItems, (seen / kItems - 1) & 1, state));
      if (!ok) break;
      if (lane == 0) {
        volatile int* to = reinterpret_cast<volatile int*>(smem + C::kOffItem + seen % kItems * 64);
        const int* from = reinterpret_cast<const int*>(&it);
#pragma unroll
        for (int e = 0; e < (int)(sizeof(Item) / 4); ++e) to[e] = from[e];
        mbar_arrive(item_full + seen % kItems);
      }
      __syncwarp();
      ++seen;
      if (it.b < 0) break;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        if (it.n[t] == 0 || (t == 1 && it.split)) continue;
        const int y = it.q0 + it.first + t * p.tpt;
        if (lane < D / 64) tma_3d_prefetch(&map_q, 64 * lane, it.hq0, y);
        if (qn[t] > 0) ok = ok && __all_sync(~0u, bar_wait(q_free + t, (qn[t] - 1) & 1, state));
        if (!ok) break;
        ++qn[t];
        if (lane == 0) {
          mbar_expect_tx(q_full + t, (uint32_t)(p.hg * p.tpt * D * 2));
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c)
            tma_3d(qs + t * C::kQ + c * kRows * 128, &map_q, 64 * c, it.hq0, y, q_full + t);
        }
        __syncwarp();
      }
    }
    for (int t = 0; t < kTiles; ++t)  // the copies land before the CTA ends
      if (qn[t] > 0) static_cast<void>(mbar_wait(q_full + t, (qn[t] - 1) & 1, nullptr));
  } else if (warp >= kFeed && warp < kMma) {
    // ---- K and V tiles through the ring in the order of their use: K_0 V_0 K_1 V_1 ..., or
    // with one Q tile K_0 K_1 V_0 K_2 V_1 ...  A warp has kMine keys of each tile, as many of
    // each half (a lane finds the page of one), of a V unit of 64 keys those ---------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsFeed));
    constexpr int kRowBytes = D * (kI8 ? 1 : 2);       // of a cached row
    constexpr int kSrcCols = C::kCols * (kI8 ? 1 : 2);  // bytes of a row in a K unit
    const int w = warp - kFeed;
    constexpr int kMine = kKeys / C::kFeeds, kHalf = kMine / 2;
    constexpr int kUnitSh = C::kCols == 128;  // a unit is 64 << kUnitSh columns (V of 256 twice that)
    const int key = 64 * (lane / kHalf & 1) + kHalf * w + lane % kHalf;
    const uint32_t stage = smem_addr(smem + C::kOffStage) + w * (C::kStage / C::kFeeds);
    uint32_t* bads = reinterpret_cast<uint32_t*>(smem + C::kOffBad) + 16 * w;
    int u = 0, f = 0;     // units issued, units handed over
    uint32_t kinds = 0;   // of the last 16 units: 1 V, 2 its second unit
    int tiles_in = 0, tiles_out = 0;  // K tiles issued, handed over
    int64_t rows[2] = {};  // this lane's row of the cache in tiles j and j - 1 (those whose V is to come)
    int page = 0;          // and its page of tile j + 1
    // Unit f has landed (its group has been waited for): to the tensor core.
    auto hand_over = [&] {
      const int at16 = f & 15, st = f % C::kRing;
      const bool v = kinds >> (2 * at16) & 1, second = kinds >> (2 * at16) & 2;
      const uint32_t to = ring + st * C::kUnit;
      __syncwarp();
      // Whatever became of a wait, all lanes go the same way, inside the ring, until the loop's end (with
      // a way out here 8192 tokens of 4 x 6 heads of 256, int8, take 1398 us for 1226).
      if constexpr (!kI8) ok = __all_sync(~0u, ok);
      if constexpr (kI8) {
        if (f >= C::kRing) ok = bar_wait(empty + st, (f / C::kRing - 1) & 1, state);
        ok = __all_sync(~0u, ok);
        const uint32_t from = stage + (f % C::kAhead) * C::kStage;
        // Eight rows and 64 codes of each at a time: four lanes a row write pieces 0, 2, 4, 6
        // of 128 bytes, then 1, 3, 5, 7, the rows beside them the others (by the swizzle).
        auto go = [&](int sh) {  // 64 << sh columns
          constexpr int kIts = C::kStage / C::kFeeds / 512, kBatch = kIts < 4 ? kIts : 4;
          const uint32_t at = to + (kHalf * w + (lane >> 2)) * 128, p0 = ((2 * (lane & 3)) ^ (lane >> 2)) << 4;
#pragma unroll
          for (int i0 = 0; i0 < kIts; i0 += kBatch) {
            uint32_t x[kBatch][4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                           : "r"(from + ((i0 + i) * 32 + lane) * 16));
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int g = (i0 + i) >> sh, block = (i0 + i) & ((1 << sh) - 1);  // rows 8 g .. of the warp
              const uint32_t d = at + block * (C::kUnit >> sh) + (64 * (8 * g / kHalf) + 8 * g % kHalf) * 128;
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) y[2 * e] = codes<0x4140>(x[i][e]), y[2 * e + 1] = codes<0x4342>(x[i][e]);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d + p0), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                           "r"(y[3])
                           : "memory");
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d + (p0 ^ 16)), "r"(y[4]), "r"(y[5]), "r"(y[6]),
                           "r"(y[7])
                           : "memory");
            }
          }
        };
        go(kUnitSh + (D == 256 && v));
        if (!v && !second) {  // this lane's scales
          const int slot = tiles_out & (kScales - 1);
          float* sc = reinterpret_cast<float*>(smem + C::kOffScale) + slot * 2 * kKeys + key;
          bool odd = false;
          if (lane < kMine) {
            if (p.key_up != 1.0f) sc[0] *= p.key_up;
            if (bads[at16] >> lane & 1) sc[0] = __int_as_float(0x7fc00000);
            odd = !(fabsf(sc[kKeys]) < -kNegInf);
            if (odd) sc[kKeys] = 0.0f;
          }
          const unsigned odds = __ballot_sync(~0u, odd);
          uint8_t* mask = smem + C::kOffOdd + slot * 16;  // (eight keys a byte)
          if (lane == 0) mask[w] = (uint8_t)odds, mask[8 + w] = (uint8_t)(odds >> 8);
          __syncwarp();
          if (lane == 0) mbar_arrive(scales + slot);
        }
      } else if (!v && !second && ok && bads[at16]) {  // a key of no page: its scores are NaN
        if (bads[at16] >> lane & 1)
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + key * 128 + ((key & 7) << 4)), "h"((short)0x7fc0) : "memory");
      }
      if (!v && !second) ++tiles_out;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0 && (kI8 || ok)) mbar_arrive(full + st);
      ++f;
    };
    // Of the unit's rows, idx / chunks is the row of this warp and idx % chunks the piece.
    auto issue = [&](bool v, int k, int64_t row) {
      const int at16 = u & 15;
      kinds = (kinds & ~(3u << (2 * at16))) | ((v ? 1u : 0u) | (k ? 2u : 0u)) << (2 * at16);
      const char* base = static_cast<const char*>(v ? a.c.v : a.c.k) + (v ? 0 : k * kSrcCols);
      if constexpr (kI8) {
        const uint32_t to = stage + (u % C::kAhead) * C::kStage;
        if (!v && k == 0) {
          const int slot = tiles_in & (kScales - 1);
          const uint32_t sc = smem_addr(smem + C::kOffScale) + slot * (2 * kKeys * 4) + 4 * key;
          if (lane < kMine) {
            copy4(sc, a.c.k_scale + (row < 0 ? 0 : row), row >= 0);
            copy4(sc + 4 * kKeys, a.c.v_scale + (row < 0 ? 0 : row), row >= 0);
          }
        }
        constexpr int kIts = C::kStage / C::kFeeds / 512;
        const int sh = kUnitSh + (D == 256 && v), row0 = D == 256 && v ? kHalf * k : 0;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          const int64_t src = __shfl_sync(~0u, row, row0 + 8 * (i >> sh) + (lane >> 2));
          copy16(to + (i * 32 + lane) * 16,
                 base + (src < 0 ? 0 : src) * kRowBytes + (lane & 3) * 16 + 64 * (i & ((1 << sh) - 1)), src >= 0);
        }
      } else {
        const uint32_t to = ring + u % C::kRing * C::kUnit;
        // Four rows and 64 columns of each at a time.
        auto go = [&](auto octs_c, auto rows_c, int row0) {
          constexpr int kOcts = decltype(octs_c)::value, kUnitRows = decltype(rows_c)::value;
          constexpr int kIts = C::kUnit / C::kFeeds / 512;
          const uint32_t at = to + (kHalf * w + (lane >> 3)) * 128, p0 = ((lane & 7) ^ (lane >> 3)) << 4;
#pragma unroll
          for (int g = 0; g < kIts / kOcts; ++g) {
            const int64_t src = __shfl_sync(~0u, row, row0 + 4 * g + (lane >> 3));
            const char* from = base + (src < 0 ? 0 : src) * kRowBytes + (lane & 7) * 16;
            const uint32_t d = at + (64 * (4 * g / kHalf) + 4 * g % kHalf) * 128 + (p0 ^ (64 * (g & 1)));
#pragma unroll
            for (int o = 0; o < kOcts; ++o)
              if (ok) copy16(d + o * kUnitRows * 128, from + 128 * o, src >= 0);
          }
        };
        using std::integral_constant;
        if (D == 256 && v)
          go(integral_constant<int, D / 64>(), integral_constant<int, C::kVKeys>(), kHalf * k);
        else
          go(integral_constant<int, C::kCols / 64>(), integral_constant<int, kKeys>(), 0);
      }
      tiles_in += !v && k == 0;
      asm volatile("cp.async.commit_group;" ::: "memory");
      ++u;
    };
    // One place each for a copy and for a hand-over: their code is long.
    Item it = {};
    int x = 0, steps = 0;   // units of the item issued, all of them
    bool ending = false;
    auto token_of = [&](int j) {  // this lane's token of tile j; -1: none
      const unsigned v = (unsigned)(it.t0 + j) * kKeys + key;
      return v < (unsigned)it.nv ? (int)v + (v >= (unsigned)a.sinks ? it.skip : 0) : -1;
    };
    // (always a load into the one register, which nothing touches until the tile is issued)
    auto page_of = [&](int token) { return __ldg(a.table + it.b * a.table_width + p.by_page(max(token, 0))); };
    for (;;) {
      const bool more = x < steps;
      if (more) {
        const int y = x / C::kUnits, k = x % C::kUnits;
        const bool v = kTiles == 2 ? y & 1 : (y && !(y & 1)) || x + C::kUnits >= steps;
        if (!v && k == 0) {
          const int j = (y + 1) / 2, token = token_of(j);
          rows[1] = rows[0];
          const bool bad = token >= 0 && (unsigned)page >= (unsigned)a.c.pages;
          rows[0] = token < 0 || bad
                        ? -1
                        : ((int64_t)page * a.c.kv_heads + it.h) * p.by_page.d + (token - p.by_page(token) * p.by_page.d);
          page = page_of(token_of(min(j + 1, it.tiles - 1)));
          const unsigned any = __ballot_sync(~0u, bad);
          if (lane == 0) bads[u & 15] = any;
        }
        // (a lane whose wait ran out, now or for a unit before, copies nothing: hand_over says so for all)
        if (!kI8 && u >= C::kRing) ok = ok && bar_wait(empty + u % C::kRing, (u / C::kRing - 1) & 1, state);
        issue(v, k, kTiles == 1 && v && x + C::kUnits < steps ? rows[1] : rows[0]);
        ++x;
      } else if (!ending && (f == u || __all_sync(~0u, item_ready()))) {
        if constexpr (!kI8) {  // (units issued and not yet handed over may have run out of time)
          ok = __all_sync(~0u, ok);
          if (!ok) break;
        }
        // A read that runs out of time issues nothing any more: either the work was at its end, or
        // the products' own waits run out.  (To leave at once takes 830 us for 817 over int8.)
        ending = !read_item(it);
        x = 0, steps = ending ? 0 : 2 * C::kUnits * it.tiles;
        if (steps) page = page_of(token_of(0));
        continue;
      } else if (f == u) {
        break;
      }
      if (u - f == C::kAhead || !more) {
        if (more)
          copies_but<C::kAhead - 1>();
        else
          copies_but(u - f - 1);
        hand_over();
        if (!ok) break;
      }
    }
    copies_but<0>();  // whatever becomes of the MMAs, the copies land before the CTA ends
  } else if (warp >= kMma && warp < kMma + kTiles) {
    // ---- MMAs.  The warp stays converged and an elected lane issues each product
    // in straight-line code; with two Q tiles each has an issuing warp of its own, and
    // one waits for barriers while the other's MMAs run ----------------------------------
    const int s = warp - kMma;
    // The lanes agree on how the waits went once a tile, when its products are issued (a vote at
    // each wait took 530 us for 514 at 8192 tokens); until then all of them go the same way, and
    // one that ran out of time issues nothing.
    auto wait = [&](uint64_t* bar, int phase) { ok = ok && bar_wait(bar, phase & 1, state); };
    auto agree = [&] {
      ok = __all_sync(~0u, ok);
    };
    // of the items before: units in the ring, tiles of this S, rounds of turns, outputs of
    // this S, Q tiles loaded
    unsigned units = 0;
    int done = 0, rounds = 0, outs = 0, qn[2] = {};
    Item it;
    while (read_item(it)) {
      const int tiles = s ? it.n[1] : it.n[0], theirs = s ? it.n[0] : it.n[1];
      if (it.tiles == 0) continue;
      const bool split = kTiles == 2 && it.split;
      const int most = split ? tiles : max(tiles, theirs), q_at = split ? 0 : s;
      qn[0] += split || it.n[0] > 0;
      qn[1] += !split && it.n[1] > 0;
      auto slot_of = [&](int j) { return kTiles == 1 ? (done + j) & 1 : s; };
      auto use_of = [&](int j) { return kTiles == 1 ? (done + j) >> 1 : done + j; };
      // the first ring unit of this S's K or V tile j
      auto k_unit = [&](int j) {
        return units + (kTiles == 1 ? 2 * (j ? 2 * j - 1 : 0) : split ? 4 * j + 2 * s : 2 * j);
      };
      auto v_unit = [&](int j) {
        return units + (kTiles == 1 ? 2 * (j + 1 < tiles ? 2 * j + 2 : 2 * j + 1) : split ? 4 * j + 2 * s + 1 : 2 * j + 1);
      };
      auto place = [&](unsigned x) { return (int)(x % C::kRing); };
      auto landed = [&](unsigned x) { wait(full + place(x), (int)(x / C::kRing)); };
      // A K or V tile that the other S does not use is released for both, but for the item's
      // last: its V both release, so that neither is more than kRing units behind the other or
      // ahead (a barrier tells one phase from the next, not from the one after).
      const bool owns_last = split ? ((it.tiles - 1) & 1) == s : tiles == most;
      auto release = [&](int j, int st, bool v) {
        mma_commit(empty + st);
        if (kTiles == 2 && (split || j >= theirs) && !(v && owns_last && j == tiles - 1)) mma_commit(empty + st);
      };
      // S of tile j into its slot; `there`: K has landed
      const uint32_t q_desc = tile_desc(qs + q_at * C::kQ, 16);
      auto scores = [&](int j, unsigned x, bool there) {
        const int slot = slot_of(j);
        if (j == 0) wait(q_full + q_at, qn[q_at] - 1);
#pragma unroll
        for (int k = 0; k < C::kUnits; ++k, ++x) {  // by columns
          const int st = place(x);
          if (!there) landed(x);
          fence_after();
          if (elected() && ok) {
            const uint32_t qd = q_desc + k * (C::kCols / 64) * (kRows * 128 / 16);
            const uint32_t kd = tile_desc(ring + st * C::kUnit, 16);
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
            release(j, st, false);
            if (k == C::kUnits - 1) {
              mma_commit(s_full + slot);
              if (j == tiles - 1) {
                mma_commit(q_free + q_at);
                if (kTiles == 2 && !split) mma_commit(q_free + q_at);
              }
            }
          }
          __syncwarp();
        }
      };
      if (split && tiles == 0) {  // (it releases the Q tile too, as above)
        wait(q_full, qn[0] - 1);
        agree();
        if (ok && lane == 0) mbar_arrive(q_free);
        __syncwarp();
      }
      if (!kAfter) scores(0, k_unit(0), false);
#pragma unroll 1
      for (int j = kAfter ? -1 : 0; j < most && ok; ++j) {
        const bool mine = j >= 0 && j < tiles, more = j + 1 < tiles;
        const unsigned k_at = k_unit(j + 1);
        if (!kAfter && more) scores(j + 1, k_at, false);
        // O += P V, over the first and second 64 keys
        const int slot = slot_of(j), use = use_of(j);
        const unsigned v = v_unit(j);
        const int v_st[2] = {place(v), place(v + C::kUnits - 1)};
        const uint32_t v_desc[2] = {tile_desc(ring + v_st[0] * C::kUnit, C::kVKeys * 128),
                                    tile_desc(ring + v_st[1] * C::kUnit + (C::kUnits == 2 ? 0 : 8192), C::kVKeys * 128)};
        if (mine) {
#pragma unroll
          for (int k = 0; k < C::kUnits; ++k) landed(v + k);
          if (j == 0 && outs > 0) wait(o_free + s, outs - 1);
        }
        // (not where S have each their own tiles: K may wait for V's release)
        const bool there = kAfter && !split && j >= 0 && more;
        if (there) landed(k_at);
#pragma unroll
        for (int half = 0; half < 2 && j >= 0; ++half) {
          if (mine) wait(p_full + 2 * slot + half, use);
          // Two Q tiles take turns: issued side by side their MMAs would alternate,
          // both S would arrive together and the tensor core would stand still
          // during both softmaxes.
          if (kAfter && half == 0 && !split) {
            const int t = rounds + j - (s == 0);
            if (t >= 0) wait(turn + s, t);
          }
          if (!mine) break;
          fence_after();
          if (elected() && ok) {
            const int st = v_st[half];
            const uint32_t pa = tmem + slot * kKeys + 32 * half;
            const uint32_t d = tmem + 2 * kKeys + s * D;
            const uint32_t vd = v_desc[half];
            if (half > 0 || j > 0)
              mma_ts<true>(d, pa, vd, idesc<D, true>());
            else
              mma_ts<false>(d, pa, vd, idesc<D, true>());
#pragma unroll
            for (int e = 1; e < 4; ++e)  // 16 keys: 8 columns of P, 2048 bytes of V
              mma_ts<true>(d, pa + 8 * e, vd + 128 * e, idesc<D, true>());
            if (half == 1 || C::kUnits == 2) release(j, st, true);
            if (half == 1) {
              if (kTiles == 1) mma_commit(pv_done + s);
              if (j == tiles - 1) mma_commit(o_full + s);
            }
          }
          __syncwarp();
        }
        if (kAfter && more) scores(j + 1, k_at, there);
        if (kAfter && !split && j >= 0 && ok && lane == 0) mbar_arrive(turn + 1 - s);
        agree();
      }
      if (kTiles == 2 && !owns_last) {
        const unsigned last = units + 2 * it.tiles - 1;
        landed(last);
        agree();
        if (ok && lane == 0) mbar_arrive(empty + place(last));
        __syncwarp();
      }
      if (!ok) break;
      done += tiles;
      if (!split) rounds += most;
      outs += tiles > 0;
      units += 2 * C::kUnits * it.tiles;
    }
    if (elected()) mma_commit(all_done);
    __syncwarp();
  } else if (warp < C::kSoftmax) {
    // ---- softmax: thread = row of its S; then the output, O over its sum -----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int s = kTiles == 1 ? 0 : warp >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int row = 32 * quarter + lane;
    const float scale2 = kI8 ? p.scale2 : a.scale * kLog2e;  // (read alone over bf16: at head_dim 256 719 us for 707)
    const uint32_t o_at = tmem + lanes + 2 * kKeys;
    // this row's token of the tile, and those of the warp's first and last row
    const int my_tok = p.by_hg(row), tok_lo = p.by_hg(32 * quarter), tok_hi = p.by_hg(32 * quarter + 31);
    const int my_head = row - my_tok * p.hg;
    float2* sums = reinterpret_cast<float2*>(smem + C::kOffSums);
    int done = 0, fed = 0, outs[2] = {}, joins = 0;  // of the items before: tiles of this S, all tiles, outputs, sums
    for (;; item_done()) {
      // The item stays where it is and is read again for the output: the registers are
      // the scores'.
      const volatile Item& it = *item_there();
      if (!ok || it.b < 0) break;
      const bool split = kTiles == 2 && it.split;
      const int tiles = s ? it.n[1] : it.n[0], t0 = it.t0;
      auto first_of = [&] { return it.first + (split ? 0 : s * p.tpt); };
      // What the row of token t sees of the run's tokens.
      auto sight_of = [&](int t) {
        const int nq = it.nq, skip = it.skip;
        const int end = max(0, it.nk - nq + min(first_of() + t, nq - 1) + 1);  // (no more than the last query)
        Sight x;
        x.sinks = a.sinks;
        x.from = a.window ? max(0, end - a.window) - skip : 0;
        x.end = end - skip;
        return x;
      };
      const Sight sight = sight_of(my_tok);
      // of the warp's rows: the first end, the last one, the last beginning
      const int lowest_end = sight_of(tok_lo).end, highest_end = sight_of(tok_hi).end, highest_from = sight_of(tok_hi).from;
      const bool idle = first_of() + tok_lo >= it.nq || 32 * quarter >= p.hg * p.tpt;  // no row of the warp is one
      float m = kNegInf;  // what P refers to, in units of log2
      bool ready = false, odd = false;
      uint64_t sum2[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
      for (int i = 0; i < tiles && ok; ++i) {
        const int g = done + i, slot = kTiles == 1 ? g & 1 : s, use = kTiles == 1 ? g >> 1 : g;
        const int j = split ? 2 * i + s : i;  // of the part's tiles
        const uint32_t at = tmem + lanes + slot * kKeys;
        ok = __all_sync(~0u, ready || bar_wait(s_full + slot, use & 1, state));
        if (!ok) break;
        if (idle) {
          if (lane == 0) {
            mbar_arrive(p_full + 2 * slot);
            mbar_arrive(p_full + 2 * slot + 1);
          }
          ready = false;
          continue;
        }
        const int v0 = (t0 + j) * kKeys;
        uint32_t ks = 0, vs = 0;  // where the tile's scales are
        if constexpr (kI8) {
          const int sc = (fed + j) & (kScales - 1);
          ok = __all_sync(~0u, bar_wait(scales + sc, ((fed + j) / kScales) & 1, state));
          if (!ok) break;
          ks = smem_addr(smem + C::kOffScale) + sc * 2 * kKeys * 4;
          vs = ks + kKeys * 4;
          const uint4 om = *reinterpret_cast<const uint4*>(smem + C::kOffOdd + sc * 16);
          if (__builtin_expect(om.x | om.y | om.z | om.w, 0)) {
            const uint32_t o[4] = {om.x, om.y, om.z, om.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int x = v0 + 32 * c;
              odd |= (o[c] & low_bits(sight.end - x) & (~low_bits(sight.from - x) | low_bits(sight.sinks - x))) != 0;
            }
          }
        }
        fence_after();
        const int left_hi = highest_end - v0;
        if (__builtin_expect(lowest_end - v0 < kKeys || (highest_from > v0 && sight.sinks - v0 < kKeys), 0)) {
          // Keys that a row does not see, in TMEM: a loop that fits the instruction cache.
#pragma unroll 1
          for (int c = 0; c < (left_hi > 64 ? kKeys : 64); c += 32) {
            const int x0 = v0 + c;
            const uint32_t in = low_bits(sight.end - x0) & (~low_bits(sight.from - x0) | low_bits(sight.sinks - x0));
            if (!kI8 && __all_sync(~0u, in == ~0u)) continue;
            uint32_t x[32];
            tmem_ld32(at + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float k[4];
              if constexpr (kI8) shared4(ks + 4 * (c + e), k);
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                if constexpr (kI8) x[e + f] = __float_as_uint(__uint_as_float(x[e + f]) * k[f]);
                if (!(in >> (e + f) & 1)) x[e + f] = 0xff800000u;
              }
            }
            tmem_st32(at + c, x);
          }
          tmem_wait_st();
          if constexpr (kI8) ks = smem_addr(smem + C::kOffOnes);
        }
        // The second 64 columns are read twice, for the maximum and again for their
        // exponentials: 128 values held beside P's do not fit the registers.
        uint32_t v[64];
        auto read_s = [&](uint32_t* to, int c0) {
          tmem_ld32(at + c0, to);
          tmem_ld32(at + c0 + 32, to + 32);
        };
        auto scaled = [&](uint32_t* x, int c0, auto n) {  // n scores of int8 codes
          if constexpr (kI8) {
#pragma unroll
            for (int e = 0; e < decltype(n)::value; e += 4) {
              float k[4], y0, y1;
              shared4(ks + 4 * (c0 + e), k);
              unpair(mul2(pair(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), pair(k[0], k[1])), y0, y1);
              x[e] = __float_as_uint(y0), x[e + 1] = __float_as_uint(y1);
              unpair(mul2(pair(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), pair(k[2], k[3])), y0, y1);
              x[e + 2] = __float_as_uint(y0), x[e + 3] = __float_as_uint(y1);
            }
          }
        };
        float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
        using std::integral_constant;
        constexpr integral_constant<int, 64> k64;
        constexpr integral_constant<int, 32> k32;
        auto take_max = [&](const uint32_t* x, auto n) {
#pragma unroll
          for (int c = 0; c < decltype(n)::value; c += 2)
            top[c / 2 % 4] = max3(top[c / 2 % 4], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        };
        if constexpr (kI8) {  // (with their scales 128 values do not fit)
          read_s(v, 0);
          tmem_wait_ld();
          scaled(v, 0, k64);
          take_max(v, k64);
          if (left_hi > 64) {
#pragma unroll
            for (int c = 64; c < kKeys; c += 32) {
              uint32_t x[32];
              tmem_ld32(at + c, x);
              tmem_wait_ld();
              scaled(x, c, k32);
              take_max(x, k32);
            }
          }
        } else {
          uint32_t second[64];
          read_s(v, 0);
          read_s(second, 64);
          tmem_wait_ld();
          take_max(v, k64);
          if (left_hi > 64) take_max(second, k64);
        }
        const float t2 = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale2;
        if (i == 0) {
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
            tmem_ld32(o_at + s * D + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_at + s * D + c, o);
          }
        }
        const float z = m == kNegInf ? 0.0f : -m;
        const uint64_t zz = pair(z, z), ss = pair(scale2, scale2);
        auto half_p = [&](int half) {  // of v
          uint32_t x[32];
          float w[4];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            unpair(fma2(pair(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), ss, zz), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum2[e & 1] = add2(sum2[e & 1], pair(x0, x1));
            if constexpr (kI8) {
              if (e % 2 == 0) shared4(vs + 4 * (64 * half + 2 * e), w);
              unpair(mul2(pair(x0, x1), pair(w[2 * (e & 1)], w[2 * (e & 1) + 1])), x0, x1);
            }
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
        // The product with V starts on the first half.
        half_p(0);
        publish(0);
        {  // whether the next S has arrived: asked now, used at the top
          const int ng = g + 1, nslot = kTiles == 1 ? ng & 1 : s, nuse = kTiles == 1 ? ng >> 1 : ng;
          ready = i + 1 < tiles && mbar_test(s_full + nslot, nuse & 1);
        }
        if (left_hi > 64) {
          read_s(v, 64);
          tmem_wait_ld();
          scaled(v, 64, k64);
          half_p(1);
        } else {
          const uint32_t none[32] = {};
          tmem_st32(at + 32, none);
        }
        publish(1);
      }
      if (!ok) break;
      done += tiles;
      const int part_tiles = it.tiles, n0 = it.n[0], n1 = it.n[1];
      fed += part_tiles;

      // ---- the output -------------------------------------------------------------------
      float l;
      {
        float lo, hi;
        unpair(add2(sum2[0], sum2[1]), lo, hi);
        l = lo + hi;
      }
      const bool two = split && n1 > 0;  // both O are one run's
      if (two && s == 1) {
        if (joins > 0) ok = __all_sync(~0u, bar_wait(ml_free, (joins - 1) & 1, state));
        if (!ok) break;
        sums[row] = make_float2(m, odd ? -l : l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
      }
      const int t = first_of() + my_tok, nq = it.nq;
      if ((split && s == 1) || (!split && t - my_tok >= nq)) {
        outs[0] += n0 > 0, outs[1] += n1 > 0, joins += two;
        continue;
      }
      float w0 = kI8 ? kCodeUp : 1.0f, w1 = 0.0f, l1 = 0.0f;
      const float l0 = l;
      if (two) {
        ok = __all_sync(~0u, bar_wait(ml_full, joins & 1, state));
        if (!ok) break;
        const float2 other = sums[row];
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_free);
        odd |= other.y < 0.0f;
        l1 = fabsf(other.y);
        const float top = fmaxf(m, other.x);
        w0 = weight(m, l0, top), w1 = weight(other.x, l1, top);
        l = l0 * w0 + l1 * w1;
        m = top;
        if constexpr (kI8) w0 *= kCodeUp, w1 *= kCodeUp;
      }
      const bool mine = row < p.hg * p.tpt && t < nq;
      const int slot = it.slot;
      const int64_t out_row = (int64_t)(it.q0 + t) * a.Hq + it.hq0 + my_head;
      const bool parts = slot >= 0 && !(slot & kWhole), onto = slot >= 0 && slot & kOnto;
      const int64_t part_row = ((int64_t)blockIdx.x * 2 + (slot & 1)) * p.part_rows + (split ? 0 : s * kRows) + row;
      if (!__builtin_expect(onto, 0)) {
        if (mine) {
          if (parts)
            p.ml[part_row] = make_float2(m, l);
          else if (a.lse)
            a.lse[out_row] = l == 0.0f ? kNegInf : (m + __log2f(l)) * kLn2;
        }
        if (!parts) {
          const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
          w0 *= inv, w1 *= inv;
        }
      }
      const int o_mine = split ? 0 : s;  // the O that this warp reads first
      const bool has0 = (o_mine ? n1 : n0) > 0;
      if (has0) ok = __all_sync(~0u, bar_wait(o_full + o_mine, outs[o_mine] & 1, state));
      if (two) ok = ok && __all_sync(~0u, bar_wait(o_full + 1, outs[1] & 1, state));
      if (!ok) break;
      fence_after();
      bool fine = true, sound = l == l;  // the output is finite; its sum is no NaN
      if (!idle) {
        const unsigned how = (two ? 1u : 0u) | (mine ? 2u : 0u) | (parts ? 4u : 0u) | (odd ? 8u : 0u) |
                             (has0 && l0 != 0.0f ? 16u : 0u) | (two && l1 != 0.0f ? 32u : 0u);
        if (__builtin_expect(onto, 0)) {
          const unsigned is = put_row_onto<D, kI8>(p, o_at + o_mine * D, o_at + D, w0, w1, m, l, how, part_row, out_row);
          fine = is & 1, odd = is & 2, sound = is & 4;
        } else {
          fine = put_row<D>(o_at + o_mine * D, o_at + D, w0, w1,
                            parts ? reinterpret_cast<char*>(p.part + part_row * D) : reinterpret_cast<char*>(a.out + out_row * D),
                            how);
        }
      }
      // the next item's products may come
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (has0) mbar_arrive(o_free + o_mine);
        if (two) mbar_arrive(o_free + 1);
      }
      outs[0] += n0 > 0, outs[1] += n1 > 0, joins += two;
      // rows whose sum is finite and whose output is not
      const unsigned again = __ballot_sync(~0u, mine && !odd && !fine && sound);
      if (__builtin_expect(again, 0)) {
        __syncwarp();
        const int n = split ? part_tiles : s ? n1 : n0;
        Item copy;
        copy.b = it.b, copy.h = it.h, copy.skip = it.skip;
        repair<D, kI8>(p, copy, again, out_row, sight, it.r0 * kKeys, min((int)it.nv, (t0 + n) * kKeys),
                       parts ? p.part + part_row * D : nullptr, p.ml + part_row, state);
      }
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

// Joins the parts of the run that begins in CTA blockIdx.x and goes on in the CTAs
// after it, in their order: a warp a row.
constexpr int kJoinCtas = 16;
template <int D>
__global__ void __launch_bounds__(256) attn_chunk_join_kernel(Args p) {
  constexpr int N = D / 32;
  pdl_release();
  pdl_wait();
  const ChunkArgs& a = p.a;
  const Note note = p.note[blockIdx.x];
  const int lane = threadIdx.x & 31, parts = note.last - (int)blockIdx.x + 1;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < note.tokens * p.hg; r += 8 * gridDim.y) {
    const int t = p.by_hg(r), head = r - t * p.hg;
    const int tile = t / p.tpt, in_part = tile * kRows + (t - tile * p.tpt) * p.hg + head;
    auto row_of = [&](int i) {
      return ((int64_t)(blockIdx.x + i) * 2 + (i ? 0 : note.slot)) * p.part_rows + in_part;
    };
    float top = kNegInf;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.ml[row_of(i)].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, i));
    float l = 0.0f;
    for (int i = lane; i < parts; i += 32) {
      const float2 ml = p.ml[row_of(i)];
      l += ml.y * weight(ml.x, ml.y, top);
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(~0u, l, i);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    float o[N] = {};
    for (int i0 = 0; i0 < parts; i0 += 32) {  // the weights of 32 parts, a lane each
      float w = 0.0f;
      if (i0 + lane < parts) {
        const float2 ml = p.ml[row_of(i0 + lane)];
        w = weight(ml.x, ml.y, top) * inv;
        if (ml.y == 0.0f) w = -1.0f;  // no key: its sums were not written
      }
      const int n = min(32, parts - i0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(~0u, w, i);
        const float* from = p.part + row_of(i0 + i) * D + lane * N;
        float x[N];
        if constexpr (N == 2) {
          const float2 v = *reinterpret_cast<const float2*>(from);
          x[0] = v.x, x[1] = v.y;
        } else {
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(from + e);
            x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (wi != -1.0f) o[e] = fmaf(wi, x[e], o[e]);
      }
    }
    const int64_t row = note.row + (int64_t)t * a.Hq + head;
    if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? kNegInf : top * kLn2 + logf(l);
#pragma unroll
    for (int i = 0; i < N; i += 2)
      *reinterpret_cast<uint32_t*>(a.out + row * D + lane * N + i) = bf16x2(o[i], o[i + 1]);
  }
}

struct Plan {
  int hg, tpt, part_rows;
};

Plan plan_of(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D) {
  Plan r;
  const int tiles = D == 256 ? 1 : 2;
  r.hg = heads_of_tile(Hq / Hkv, B, Tq, tiles);
  r.tpt = kRows / r.hg;
  r.part_rows = Tq <= r.tpt ? (int)Tq * r.hg : tiles * kRows;  // one tile, as far as it is filled
  return r;
}

size_t workspace_of(const Plan& r, int64_t D) {
  return (size_t)kCtas * (2 * (size_t)r.part_rows * (size_t)(D * 4 + 8) + sizeof(Note)) + 768;
}

template <int D, bool kI8>
cudaError_t launch(const ChunkArgs& a, void* ws, cudaStream_t st) {
  using C = Cfg<D, kI8>;
  const Plan plan = plan_of(a.B, a.Tq, a.Hq, a.c.kv_heads, D);
  const int64_t G = a.Hq / a.c.kv_heads;
  Args p{a, (int)G, plan.hg, plan.tpt, (int)(a.c.kv_heads * (G / plan.hg)), C::kTiles * plan.tpt, plan.part_rows,
         Divider(G), Divider(plan.hg), Divider(C::kTiles * plan.tpt), Divider(a.c.page_tokens), a.scale * kLog2e, 1.0f, nullptr, nullptr, nullptr};
  if (kI8) (a.scale < 0x1p100f ? p.scale2 : p.key_up) *= kCodeUp;
  auto up = [](void* q) { return (reinterpret_cast<uintptr_t>(q) + 255) & ~(uintptr_t)255; };
  const size_t rows = (size_t)kCtas * 2 * plan.part_rows;
  p.part = reinterpret_cast<float*>(up(ws));
  p.ml = reinterpret_cast<float2*>(up(p.part + rows * D));
  p.note = reinterpret_cast<Note*>(up(p.ml + rows));
  CUtensorMap mq;
  cudaError_t e = encode_tma_heads(&mq, a.q, D, a.Hq, a.Tq, a.q_stride, p.hg, p.tpt);
  if (e != cudaSuccess) return e;
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidDevice;
  auto kern = attn_chunk_kernel<D, kI8>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(kCtas), dim3(C::kThreads), C::kSmem, st, mq, p, status);
  if (e != cudaSuccess) return e;
  const int y = (plan.part_rows + 7) / 8;
  return launch_pdl(attn_chunk_join_kernel<D>, dim3(kCtas, y < kJoinCtas ? y : kJoinCtas), dim3(256), 0, st, p);
}

template <bool kI8>
cudaError_t by_dim(const ChunkArgs& a, void* ws, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch<64, kI8>(a, ws, st);
    case 128: return launch<128, kI8>(a, ws, st);
    default: return launch<256, kI8>(a, ws, st);
  }
}

}  // namespace

size_t attn_chunk_workspace(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Tq == 0) return 0;
  return workspace_of(plan_of(B, Tq, Hq, Hkv, D), D);
}

cudaError_t launch_attn_chunk(const ChunkArgs& a, void* ws, cudaStream_t st) {
  return a.c.type == PTQ_KV_I8 ? by_dim<true>(a, ws, st) : by_dim<false>(a, ws, st);
}

}  // namespace ptq
