// api_attn.cu -- the C ABI of the paged key-value cache and the attention
// over it: argument validation, then one launcher each.  Every entry point
// validates everything before it launches anything.
#include <math.h>

#include "ptq_internal.cuh"

using namespace ptq;

namespace {

bool head_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

// A strided token matrix: rows of `row` elements, `stride` elements apart.
bool stride_ok(int64_t stride, int64_t row, int64_t tokens, ptq_dtype dt) {
  int64_t t;
  return stride >= row && mul_ok(tokens, stride, &t) && mul_ok(t, (int64_t)dsize(dt), &t);
}

bool stride_aligned(int64_t stride, ptq_dtype dt) { return stride * (int64_t)dsize(dt) % 16 == 0; }

ptq_status check_cache(const ptq_kv_cache* c, const char* who) {
  if (!c) return fail(PTQ_ERR_NULL, "%s: cache is NULL", who);
  if (c->type != PTQ_KV_BF16 && c->type != PTQ_KV_I8)
    return fail(PTQ_ERR_VALUE, "%s: unknown cache type %d", who, (int)c->type);
  int64_t slots, t;
  if (c->pages < 1 || c->page_tokens < 1 || c->kv_heads < 1 || c->head_dim < 1 ||
      c->kv_heads > INT32_MAX || !mul_ok(c->pages, c->page_tokens, &slots) || slots > INT32_MAX ||
      !mul_ok(slots, c->kv_heads, &t) || !mul_ok(t, c->head_dim, &t) || !mul_ok(t, 2, &t))
    return fail(PTQ_ERR_SHAPE,
                "%s: need pages, page_tokens, kv_heads >= 1 and under 2^31 slots (pages=%lld "
                "page_tokens=%lld kv_heads=%lld head_dim=%lld)", who, (long long)c->pages,
                (long long)c->page_tokens, (long long)c->kv_heads, (long long)c->head_dim);
  if (!head_dim_ok(c->head_dim))
    return fail(PTQ_ERR_UNSUPPORTED, "%s: head_dim is 64, 128 or 256, got %lld", who,
                (long long)c->head_dim);
  if (!c->k || !c->v || (c->type == PTQ_KV_I8 && (!c->k_scale || !c->v_scale)))
    return fail(PTQ_ERR_NULL, "%s: NULL pointer in the cache", who);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) ||
      (c->type == PTQ_KV_I8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
    return fail(PTQ_ERR_ALIGN, "%s: the cache's k and v need 16-byte, its scales 4-byte alignment",
                who);
  return PTQ_OK;
}

ptq_status check_rows(const ptq_kv_cache* c, const void* k, const void* v, int64_t k_stride,
                      int64_t v_stride, const int32_t* slots, int64_t T, ptq_dtype dt,
                      const char* who) {
  if (!dtype_ok(dt)) return fail(PTQ_ERR_VALUE, "%s: unknown dtype %d", who, (int)dt);
  const ptq_status s = check_cache(c, who);
  if (s != PTQ_OK) return s;
  const int64_t row = c->kv_heads * c->head_dim;
  if (T < 0 || T > INT32_MAX || !stride_ok(k_stride, row, T, dt) || !stride_ok(v_stride, row, T, dt))
    return fail(PTQ_ERR_SHAPE,
                "%s: need 0 <= T < 2^31 and strides of at least kv_heads * head_dim (T=%lld "
                "strides=%lld, %lld)", who, (long long)T, (long long)k_stride, (long long)v_stride);
  if (T == 0) return PTQ_OK;
  if (!k || !v || !slots) return fail(PTQ_ERR_NULL, "%s: NULL pointer", who);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !stride_aligned(k_stride, dt) ||
      !stride_aligned(v_stride, dt))
    return fail(PTQ_ERR_ALIGN,
                "%s: k, v and their strides need 16-byte, slots 4-byte alignment", who);
  return PTQ_OK;
}

bool heads_ok(int64_t Hq, int64_t Hkv) {
  return Hkv >= 1 && Hq >= Hkv && Hq <= INT32_MAX && Hq % Hkv == 0;
}

ptq_status check_scale(float scale, const char* who) {
  if (!(scale > 0.0f) || !(scale < INFINITY))
    return fail(PTQ_ERR_VALUE, "%s: softmax_scale must be finite and positive", who);
  return PTQ_OK;
}

ptq_status check_window(int64_t window, int64_t sinks, const char* who) {
  if (window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX)
    return fail(PTQ_ERR_VALUE, "%s: window and sinks are 0 to 2^31 - 1 (%lld, %lld)", who,
                (long long)window, (long long)sinks);
  return PTQ_OK;
}

// The head norms and rotation of T tokens whose heads are D wide.
ptq_status check_rope(const ptq_rope* r, int64_t T, int64_t D, ptq_dtype dt, const char* who) {
  if (!r) return fail(PTQ_ERR_NULL, "%s: rope is NULL", who);
  if (!dtype_ok(dt)) return fail(PTQ_ERR_VALUE, "%s: unknown dtype %d", who, (int)dt);
  int64_t t;
  if (r->rotary_dim < 0 || r->rotary_dim > D || r->rotary_dim % 8 != 0 ||
      (r->rotary_dim > 0 && (r->axes < 1 || r->axes > 127 || (r->axes > 1 && r->pos_stride < T) ||
                             !mul_ok(r->axes - 1, r->pos_stride, &t) || !mul_ok(t, 4, &t))))
    return fail(PTQ_ERR_SHAPE,
                "%s: need rotary_dim a multiple of 8 up to head_dim, 1 to 127 axes and a pos_stride of "
                "at least T (rotary_dim=%lld axes=%lld pos_stride=%lld)", who,
                (long long)r->rotary_dim, (long long)r->axes, (long long)r->pos_stride);
  if ((r->q_gain || r->k_gain) && (!(r->eps > 0.0f) || !(r->eps < INFINITY)))
    return fail(PTQ_ERR_VALUE, "%s: eps must be finite and positive", who);
  if (T > 0 && r->rotary_dim > 0 && (!r->inv_freq || !r->pos))
    return fail(PTQ_ERR_NULL, "%s: NULL pointer in rope", who);
  if (!aligned(r->q_gain, 16) || !aligned(r->k_gain, 16) || !aligned(r->inv_freq, 4) ||
      !aligned(r->pos, 4))
    return fail(PTQ_ERR_ALIGN, "%s: gains need 16-byte, inv_freq and pos 4-byte alignment", who);
  return PTQ_OK;
}

// T x heads x D values of dt, `stride` apart.
ptq_status check_heads(const void* p, int64_t stride, int64_t heads, int64_t D, int64_t T,
                       ptq_dtype dt, const char* name, const char* who) {
  if (heads == 0) return PTQ_OK;
  if (!stride_ok(stride, heads * D, T, dt))
    return fail(PTQ_ERR_SHAPE, "%s: the stride of %s is at least heads * head_dim (%lld)", who, name,
                (long long)stride);
  if (T == 0) return PTQ_OK;
  if (!p) return fail(PTQ_ERR_NULL, "%s: %s is NULL", who, name);
  if (!aligned(p, 16) || !stride_aligned(stride, dt))
    return fail(PTQ_ERR_ALIGN, "%s: %s and its stride need 16-byte alignment", who, name);
  return PTQ_OK;
}

RopeArgs rope_args(const ptq_rope& r, int64_t T, int64_t Hq, int64_t Hkv, ptq_dtype dt) {
  RopeArgs a = {};
  a.inv_freq = r.inv_freq;
  a.axis = r.axis;
  a.pos = r.pos;
  a.pos_stride = r.pos_stride;
  a.axes = (int)r.axes;
  a.rotary = (int)r.rotary_dim;
  a.near = r.interleaved != 0;
  a.q_gain = r.q_gain;
  a.k_gain = r.k_gain;
  a.eps = r.eps;
  a.T = T;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.t = act_of(dt);
  return a;
}

// Heads of a token that one call takes: their rows are counted in 32 bits.
constexpr int64_t kMostHeads = (int64_t)1 << 20;

ptq_status check_workspace(const void* ws, size_t ws_bytes, size_t need, const char* who) {
  if (need == 0) return PTQ_OK;
  if (!ws) return fail(PTQ_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", who, need);
  if (ws_bytes < need)
    return fail(PTQ_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", who, ws_bytes, need);
  if (!aligned(ws, 16)) return fail(PTQ_ERR_ALIGN, "%s: workspace needs 16-byte alignment", who);
  return PTQ_OK;
}

bool decode_shape_ok(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  int64_t t;
  return B >= 0 && B <= INT32_MAX / 2 && heads_ok(Hq, Hkv) && D >= 1 && mul_ok(B, Hq, &t) &&
         t <= INT32_MAX && mul_ok(t, D, &t) && mul_ok(t, 4, &t);
}

// Every CTA reads the sequences' offsets twice, 32 at a time: 2^26 of them take less
// than a second, well under the limit of the waits for what comes of it.
constexpr int64_t kMostPrompts = (int64_t)1 << 26;

bool prefill_shape_ok(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D) {
  int64_t t;
  return B >= 0 && B < kMostPrompts && Tq >= 0 && Tq <= INT32_MAX / 2 && Tk >= 0 &&
         Tk <= INT32_MAX / 2 && heads_ok(Hq, Hkv) && D >= 1 && mul_ok(Tq, Hq, &t) &&
         mul_ok(t, D, &t) && mul_ok(t, 4, &t);
}

ptq_status attn_decode(const void* q, int64_t q_stride, const ptq_kv_cache* cache,
                       const int32_t* table, int64_t table_width, const int32_t* lens, void* out,
                       float* lse, int64_t B, int64_t q_heads, float softmax_scale, int64_t window,
                       int64_t sinks, ptq_dtype dtype, void* ws, size_t ws_bytes,
                       ptq_stream_t stream, const char* who) {
  clear_error();
  if (!dtype_ok(dtype)) return fail(PTQ_ERR_VALUE, "%s: unknown dtype %d", who, (int)dtype);
  ptq_status s = check_cache(cache, who);
  if (s == PTQ_OK) s = check_scale(softmax_scale, who);
  if (s == PTQ_OK) s = check_window(window, sinks, who);
  if (s != PTQ_OK) return s;
  int64_t t;
  if (!decode_shape_ok(B, q_heads, cache->kv_heads, cache->head_dim) || table_width < 0 ||
      !mul_ok(table_width, cache->page_tokens, &t) || t > INT32_MAX ||
      !stride_ok(q_stride, q_heads * cache->head_dim, B, dtype))
    return fail(PTQ_ERR_SHAPE,
                "%s: need B >= 0, q_heads a multiple of kv_heads, under 2^31 tokens a table row "
                "and a stride of at least q_heads * head_dim (B=%lld q_heads=%lld kv_heads=%lld "
                "table_width=%lld q_stride=%lld)", who, (long long)B, (long long)q_heads,
                (long long)cache->kv_heads, (long long)table_width, (long long)q_stride);
  if (B == 0) return PTQ_OK;
  if (!q || !lens || !out || (!table && table_width > 0))
    return fail(PTQ_ERR_NULL, "%s: NULL pointer", who);
  if (!aligned(q, 16) || !aligned(out, 16) || !stride_aligned(q_stride, dtype) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return fail(PTQ_ERR_ALIGN,
                "%s: q, its stride and out need 16-byte, table, lens and lse 4-byte alignment", who);
  s = check_workspace(ws, ws_bytes,
                      attn_decode_workspace(B, q_heads, cache->kv_heads, cache->head_dim), who);
  if (s != PTQ_OK) return s;
  const DecodeArgs a{q, q_stride, *cache, table, table_width, lens, out, lse, B, q_heads,
                     softmax_scale, act_of(dtype), (int)window, (int)sinks};
  const cudaError_t e = launch_attn_decode(a, ws, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, who);
}

// Tokens that a query of a chunk may see: the sums of 2^12 pieces of 2^15, joined one after the other
// in fp32, are off by 2^-12 of themselves at most, an eighth of what the output is rounded by.
constexpr int64_t kMostSeen = (int64_t)1 << 27;

bool chunk_shape_ok(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D) {
  return prefill_shape_ok(B, Tq, 0, Hq, Hkv, D);
}

}  // namespace

extern "C" {

PTQ_API ptq_status ptq_kv_write(const ptq_kv_cache* cache, const void* k, const void* v,
                                int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                int64_t T, ptq_dtype dtype, ptq_stream_t stream) {
  clear_error();
  const ptq_status s =
      check_rows(cache, k, v, k_stride, v_stride, slots, T, dtype, "ptq_kv_write");
  if (s != PTQ_OK || T == 0) return s;
  const KvRows r{const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride, slots, T,
                 act_of(dtype)};
  const cudaError_t e = launch_kv_write(*cache, r, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, "ptq_kv_write launch");
}

PTQ_API ptq_status ptq_kv_read(const ptq_kv_cache* cache, const int32_t* slots, int64_t T, void* k,
                               void* v, int64_t k_stride, int64_t v_stride, ptq_dtype dtype,
                               ptq_stream_t stream) {
  clear_error();
  const ptq_status s = check_rows(cache, k, v, k_stride, v_stride, slots, T, dtype, "ptq_kv_read");
  if (s != PTQ_OK || T == 0) return s;
  const KvRows r{k, v, k_stride, v_stride, slots, T, act_of(dtype)};
  const cudaError_t e = launch_kv_read(*cache, r, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, "ptq_kv_read launch");
}

PTQ_API size_t ptq_attn_decode_workspace_bytes(int64_t B, int64_t q_heads, int64_t kv_heads,
                                               int64_t head_dim, ptq_dtype dtype) {
  if (!dtype_ok(dtype) || !decode_shape_ok(B, q_heads, kv_heads, head_dim) ||
      !head_dim_ok(head_dim))
    return 0;
  return attn_decode_workspace(B, q_heads, kv_heads, head_dim);
}

PTQ_API ptq_status ptq_attn_decode(const void* q, int64_t q_stride, const ptq_kv_cache* cache,
                                   const int32_t* table, int64_t table_width, const int32_t* lens,
                                   void* out, float* lse, int64_t B, int64_t q_heads,
                                   float softmax_scale, ptq_dtype dtype, void* ws, size_t ws_bytes,
                                   ptq_stream_t stream) {
  return attn_decode(q, q_stride, cache, table, table_width, lens, out, lse, B, q_heads,
                     softmax_scale, 0, 0, dtype, ws, ws_bytes, stream, "ptq_attn_decode");
}

PTQ_API ptq_status ptq_attn_decode_window(const void* q, int64_t q_stride,
                                          const ptq_kv_cache* cache, const int32_t* table,
                                          int64_t table_width, const int32_t* lens, void* out,
                                          float* lse, int64_t B, int64_t q_heads,
                                          float softmax_scale, int64_t window, int64_t sinks,
                                          ptq_dtype dtype, void* ws, size_t ws_bytes,
                                          ptq_stream_t stream) {
  return attn_decode(q, q_stride, cache, table, table_width, lens, out, lse, B, q_heads,
                     softmax_scale, window, sinks, dtype, ws, ws_bytes, stream,
                     "ptq_attn_decode_window");
}

PTQ_API size_t ptq_attn_prefill_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t q_heads,
                                                int64_t kv_heads, int64_t head_dim,
                                                ptq_dtype dtype) {
  if (dtype != PTQ_BF16 || !prefill_shape_ok(B, Tq, Tk, q_heads, kv_heads, head_dim) ||
      !head_dim_ok(head_dim))
    return 0;
  return attn_prefill_workspace(B, Tq, Tk, q_heads, kv_heads, head_dim);
}

PTQ_API ptq_status ptq_attn_prefill(const void* q, const void* k, const void* v, int64_t q_stride,
                                    int64_t k_stride, int64_t v_stride, const int32_t* cu_q,
                                    const int32_t* cu_k, void* out, float* lse, int64_t B,
                                    int64_t Tq, int64_t Tk, int64_t q_heads, int64_t kv_heads,
                                    int64_t head_dim, float softmax_scale, unsigned flags,
                                    ptq_dtype dtype, void* ws, size_t ws_bytes,
                                    ptq_stream_t stream) {
  clear_error();
  const char* who = "ptq_attn_prefill";
  if (!dtype_ok(dtype)) return fail(PTQ_ERR_VALUE, "%s: unknown dtype %d", who, (int)dtype);
  if (flags & ~(unsigned)PTQ_ATTN_CAUSAL)
    return fail(PTQ_ERR_VALUE, "%s: unknown flags 0x%x", who, flags);
  ptq_status s = check_scale(softmax_scale, who);
  if (s != PTQ_OK) return s;
  if (!prefill_shape_ok(B, Tq, Tk, q_heads, kv_heads, head_dim) ||
      !stride_ok(q_stride, q_heads * head_dim, Tq, dtype) ||
      !stride_ok(k_stride, kv_heads * head_dim, Tk, dtype) ||
      !stride_ok(v_stride, kv_heads * head_dim, Tk, dtype))
    return fail(PTQ_ERR_SHAPE,
                "%s: need B, Tq, Tk >= 0, q_heads a multiple of kv_heads and strides of at least a "
                "token's heads (B=%lld Tq=%lld Tk=%lld q_heads=%lld kv_heads=%lld strides=%lld, "
                "%lld, %lld)", who, (long long)B, (long long)Tq, (long long)Tk, (long long)q_heads,
                (long long)kv_heads, (long long)q_stride, (long long)k_stride, (long long)v_stride);
  if (!head_dim_ok(head_dim))
    return fail(PTQ_ERR_UNSUPPORTED, "%s: head_dim is 64, 128 or 256, got %lld", who,
                (long long)head_dim);
  if (dtype != PTQ_BF16)
    return fail(PTQ_ERR_UNSUPPORTED, "%s: no kernel for dtype=f32 (prompts are bf16)", who);
  if (B == 0 || Tq == 0) return PTQ_OK;
  if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v)))
    return fail(PTQ_ERR_NULL, "%s: NULL pointer", who);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !stride_aligned(q_stride, dtype) || !stride_aligned(k_stride, dtype) ||
      !stride_aligned(v_stride, dtype) || !aligned(cu_q, 4) || !aligned(cu_k, 4) ||
      !aligned(lse, 4))
    return fail(PTQ_ERR_ALIGN,
                "%s: q, k, v, their strides and out need 16-byte, cu_q, cu_k and lse 4-byte "
                "alignment", who);
  s = check_workspace(ws, ws_bytes,
                      attn_prefill_workspace(B, Tq, Tk, q_heads, kv_heads, head_dim), who);
  if (s != PTQ_OK) return s;
  const PrefillArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                      static_cast<const uint16_t*>(v), q_stride, k_stride, v_stride, cu_q, cu_k,
                      static_cast<uint16_t*>(out), lse, B, Tq, Tk, q_heads, kv_heads, head_dim,
                      softmax_scale, (flags & PTQ_ATTN_CAUSAL) != 0};
  const cudaError_t e = launch_attn_prefill(a, ws, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, "ptq_attn_prefill launch");
}

PTQ_API ptq_status ptq_qk_rope(const ptq_rope* rope, const void* q, const void* k, int64_t q_stride,
                               int64_t k_stride, void* q_out, void* k_out, int64_t q_out_stride,
                               int64_t k_out_stride, int64_t T, int64_t q_heads, int64_t kv_heads,
                               int64_t head_dim, ptq_dtype dtype, ptq_stream_t stream) {
  clear_error();
  const char* who = "ptq_qk_rope";
  if (T < 0 || T > INT32_MAX || q_heads < 0 || kv_heads < 0 || q_heads > kMostHeads ||
      kv_heads > kMostHeads || q_heads + kv_heads == 0 || head_dim < 1)
    return fail(PTQ_ERR_SHAPE,
                "%s: need 0 <= T < 2^31 and up to 2^20 heads (T=%lld q_heads=%lld kv_heads=%lld "
                "head_dim=%lld)", who, (long long)T, (long long)q_heads, (long long)kv_heads,
                (long long)head_dim);
  if (!head_dim_ok(head_dim))
    return fail(PTQ_ERR_UNSUPPORTED, "%s: head_dim is 64, 128 or 256, got %lld", who,
                (long long)head_dim);
  ptq_status s = check_rope(rope, T, head_dim, dtype, who);
  if (s == PTQ_OK) s = check_heads(q, q_stride, q_heads, head_dim, T, dtype, "q", who);
  if (s == PTQ_OK) s = check_heads(k, k_stride, kv_heads, head_dim, T, dtype, "k", who);
  if (s == PTQ_OK) s = check_heads(q_out, q_out_stride, q_heads, head_dim, T, dtype, "q_out", who);
  if (s == PTQ_OK) s = check_heads(k_out, k_out_stride, kv_heads, head_dim, T, dtype, "k_out", who);
  if (s != PTQ_OK || T == 0) return s;
  RopeArgs a = rope_args(*rope, T, q_heads, kv_heads, dtype);
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  a.q_stride = q_stride, a.k_stride = k_stride, a.qo_stride = q_out_stride, a.ko_stride = k_out_stride;
  const cudaError_t e = launch_rope(a, nullptr, head_dim, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, who);
}

PTQ_API ptq_status ptq_kv_append(const ptq_kv_cache* cache, const ptq_rope* rope, const void* q,
                                 const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, const int32_t* slots, void* q_out,
                                 int64_t q_out_stride, int64_t T, int64_t q_heads, ptq_dtype dtype,
                                 ptq_stream_t stream) {
  clear_error();
  const char* who = "ptq_kv_append";
  ptq_status s = check_rows(cache, k, v, k_stride, v_stride, slots, T, dtype, who);
  if (s != PTQ_OK) return s;
  const int64_t D = cache->head_dim, Hkv = cache->kv_heads;
  if (q_heads < 0 || q_heads > kMostHeads || Hkv > kMostHeads)
    return fail(PTQ_ERR_SHAPE, "%s: need up to 2^20 heads (q_heads=%lld kv_heads=%lld)", who,
                (long long)q_heads, (long long)Hkv);
  s = check_rope(rope, T, D, dtype, who);
  if (s == PTQ_OK) s = check_heads(q, q_stride, q_heads, D, T, dtype, "q", who);
  if (s == PTQ_OK) s = check_heads(q_out, q_out_stride, q_heads, D, T, dtype, "q_out", who);
  if (s != PTQ_OK || T == 0) return s;
  RopeArgs a = rope_args(*rope, T, q_heads, Hkv, dtype);
  a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.slots = slots;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.qo_stride = q_out_stride;
  a.ck = cache->k, a.cv = cache->v, a.ks = cache->k_scale, a.vs = cache->v_scale;
  const cudaError_t e = launch_rope(a, cache, D, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, who);
}

PTQ_API size_t ptq_attn_chunk_workspace_bytes(int64_t B, int64_t Tq, int64_t q_heads,
                                              int64_t kv_heads, int64_t head_dim, ptq_dtype dtype) {
  if (dtype != PTQ_BF16 || !chunk_shape_ok(B, Tq, q_heads, kv_heads, head_dim) ||
      !head_dim_ok(head_dim))
    return 0;
  return attn_chunk_workspace(B, Tq, q_heads, kv_heads, head_dim);
}

PTQ_API ptq_status ptq_attn_chunk(const void* q, int64_t q_stride, const ptq_kv_cache* cache,
                                  const int32_t* table, int64_t table_width, const int32_t* lens,
                                  const int32_t* cu_q, void* out, float* lse, int64_t B, int64_t Tq,
                                  int64_t q_heads, float softmax_scale, int64_t window,
                                  int64_t sinks, ptq_dtype dtype, void* ws, size_t ws_bytes,
                                  ptq_stream_t stream) {
  clear_error();
  const char* who = "ptq_attn_chunk";
  if (!dtype_ok(dtype)) return fail(PTQ_ERR_VALUE, "%s: unknown dtype %d", who, (int)dtype);
  ptq_status s = check_cache(cache, who);
  if (s == PTQ_OK) s = check_scale(softmax_scale, who);
  if (s == PTQ_OK) s = check_window(window, sinks, who);
  if (s != PTQ_OK) return s;
  int64_t t;
  if (!chunk_shape_ok(B, Tq, q_heads, cache->kv_heads, cache->head_dim) || table_width < 0 ||
      !mul_ok(table_width, cache->page_tokens, &t) || t > INT32_MAX ||
      !stride_ok(q_stride, q_heads * cache->head_dim, Tq, dtype))
    return fail(PTQ_ERR_SHAPE,
                "%s: need B, Tq >= 0, q_heads a multiple of kv_heads, under 2^31 tokens a table row "
                "and a stride of at least q_heads * head_dim (B=%lld Tq=%lld q_heads=%lld "
                "kv_heads=%lld table_width=%lld q_stride=%lld)", who, (long long)B, (long long)Tq,
                (long long)q_heads, (long long)cache->kv_heads, (long long)table_width,
                (long long)q_stride);
  if (dtype != PTQ_BF16)
    return fail(PTQ_ERR_UNSUPPORTED, "%s: no kernel for dtype=f32 (chunks are bf16)", who);
  if (t > kMostSeen && (window == 0 || window + sinks > kMostSeen))
    return fail(PTQ_ERR_UNSUPPORTED,
                "%s: a table row and a window of over 2^27 tokens (%lld, %lld + %lld)", who, (long long)t,
                (long long)window, (long long)sinks);
  if (B == 0 || Tq == 0) return PTQ_OK;
  if (!q || !lens || !cu_q || !out || (!table && table_width > 0))
    return fail(PTQ_ERR_NULL, "%s: NULL pointer", who);
  if (!aligned(q, 16) || !aligned(out, 16) || !stride_aligned(q_stride, dtype) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4))
    return fail(PTQ_ERR_ALIGN,
                "%s: q, its stride and out need 16-byte, table, lens, cu_q and lse 4-byte alignment",
                who);
  s = check_workspace(ws, ws_bytes,
                      attn_chunk_workspace(B, Tq, q_heads, cache->kv_heads, cache->head_dim), who);
  if (s != PTQ_OK) return s;
  const ChunkArgs a{static_cast<const uint16_t*>(q), q_stride, *cache, table, table_width, lens, cu_q,
                    static_cast<uint16_t*>(out), lse, B, Tq, q_heads, softmax_scale, (int)window,
                    (int)sinks};
  const cudaError_t e = launch_attn_chunk(a, ws, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PTQ_OK : cuda_fail(e, who);
}

}  // extern "C"
