// C ABI of the bounded-memory attention operators: argument checks and launches.
// Declarations and the contract of every entry point are in include/mka.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/mka.h"
#include "common.cuh"
#include "kernels.h"

using namespace mka;

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_last_error(code, buf);
}

#define CUDA_TRY(expr)                                                                        \
  do {                                                                                        \
    cudaError_t e_ = (expr);                                                                  \
    if (e_ != cudaSuccess) return fail(MKA_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)
#define NEED(p)                                                                                             \
  do {                                                                                                      \
    if (!(p)) return fail(MKA_ERR_INVALID_ARG, "%s: " #p " is NULL", __func__);                             \
    if ((uintptr_t)(p) & 15) return fail(MKA_ERR_INVALID_ARG, "%s: " #p " is not 16-byte aligned", __func__); \
  } while (0)
#define OPTIONAL(p) \
  do {              \
    if (p) NEED(p); \
  } while (0)

// Operands of a call, checked last: an output may not overlap another operand.  (A kernel reads positions and kept
// rows several times over; what it writes in between must not change them.)
struct Span {
  const char* name;
  const void* p;  // null: not given
  size_t bytes;
  bool out;
};
int check_apart(const char* who, std::initializer_list<Span> spans) {
  for (const Span* a = spans.begin(); a != spans.end(); ++a)
    for (const Span* b = spans.begin(); b != a; ++b)
      if ((a->out || b->out) && a->p && b->p && (uintptr_t)a->p < (uintptr_t)b->p + b->bytes &&
          (uintptr_t)b->p < (uintptr_t)a->p + a->bytes)
        return fail(MKA_ERR_INVALID_ARG, "%s: %s and %s overlap", who, b->name, a->name);
  return MKA_OK;
}
// The same for operands of `rows` rows of bf16, some elements apart: they may lie in each other's gaps.
struct RowSpan {
  const char* name;
  const void* p;
  int width, ld;
  bool out;
};
int check_rows_apart(const char* who, long long rows, std::initializer_list<RowSpan> spans) {
  for (const RowSpan* a = spans.begin(); a != spans.end(); ++a)
    for (const RowSpan* b = spans.begin(); b != a; ++b) {
      if (!a->out && !b->out) continue;
      const uintptr_t a0 = (uintptr_t)a->p, b0 = (uintptr_t)b->p;
      if (a0 >= b0 + 2 * ((rows - 1) * b->ld + b->width) || b0 >= a0 + 2 * ((rows - 1) * a->ld + a->width)) continue;
      if (a->ld == b->ld) {  // columns of one array: b's begin `gap` bytes behind a's in the row
        const uintptr_t row = 2 * (uintptr_t)a->ld, gap = (b0 % row + row - a0 % row) % row;
        if (gap >= 2 * (uintptr_t)a->width && row - gap >= 2 * (uintptr_t)b->width) continue;
      }
      return fail(MKA_ERR_INVALID_ARG, "%s: %s and %s overlap", who, b->name, a->name);
    }
  return MKA_OK;
}

// Heads, head size and scale shared by the operators' configurations.
int check_heads(const char* who, int Hq, int Hkv, int dh, float scale, float* out) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv) return fail(MKA_ERR_INVALID_ARG, "%s: n_q_heads must be a positive multiple of n_kv_heads", who);
  if (dh != 64 && dh != 128) return fail(MKA_ERR_UNSUPPORTED, "%s: d_head must be 64 or 128", who);
  if (!isfinite(scale)) return fail(MKA_ERR_INVALID_ARG, "%s: attn_scale must be finite", who);
  *out = scale > 0.f ? scale : 1.f / sqrtf((float)dh);
  return MKA_OK;
}

// ---------------------------------------------------------------- window attention
struct Win {
  int B, S, Hq, Hkv, dh, window, sinks, Spad;
  float scale;
  AttnBwdStrides ld;
};
int check_win(const char* who, const mka_attn_config* c, const mka_attn_strides* st, Win* o) {
  if (!c) return fail(MKA_ERR_INVALID_ARG, "%s: cfg is NULL", who);
  if (c->batch < 1 || c->seq < 1) return fail(MKA_ERR_INVALID_ARG, "%s: batch and seq must be >= 1", who);
  const int e = check_heads(who, c->n_q_heads, c->n_kv_heads, c->d_head, c->attn_scale, &o->scale);
  if (e != MKA_OK) return e;
  if (c->dtype == MKA_F32) return fail(MKA_ERR_UNSUPPORTED, "%s: bf16 only", who);
  if (c->dtype != MKA_BF16) return fail(MKA_ERR_INVALID_ARG, "%s: dtype must be MKA_BF16", who);
  if (c->window < 0 || c->sinks < 0) return fail(MKA_ERR_INVALID_ARG, "%s: window and sinks must be >= 0", who);
  o->B = c->batch; o->S = c->seq; o->Hq = c->n_q_heads; o->Hkv = c->n_kv_heads; o->dh = c->d_head;
  if (c->batch > 65535 || c->n_q_heads > 65535 || (long long)c->batch * c->seq > (1LL << 30) ||
      (long long)c->batch * c->n_q_heads * ((c->seq + 127) / 128) > (1LL << 30) ||
      (long long)c->n_q_heads * c->d_head > (1LL << 24))
    return fail(MKA_ERR_UNSUPPORTED, "%s: batch, seq or heads too large", who);
  // a window that reaches every earlier position is none, and without a window the sinks change nothing
  o->window = c->window >= c->seq ? 0 : c->window;
  o->sinks = o->window ? (c->sinks < c->seq ? c->sinks : c->seq) : 0;
  o->Spad = (c->seq + 127) / 128 * 128;
  const int dq = c->n_q_heads * c->d_head, dkv = c->n_kv_heads * c->d_head;
  const mka_attn_strides z = {0, 0, 0, 0, 0}, *s = st ? st : &z;
  const int want[5] = {dq, dkv, dkv, dq, dq}, got[5] = {s->q, s->k, s->v, s->out, s->dout};
  int ld[5];
  for (int i = 0; i < 5; ++i) {
    ld[i] = got[i] ? got[i] : want[i];
    if (ld[i] < want[i] || ld[i] % 8 || ld[i] > (1 << 28))
      return fail(MKA_ERR_INVALID_ARG, "%s: a row stride must be a multiple of 8 and at least the row's width", who);
  }
  o->ld = {ld[0], ld[1], ld[2], ld[3], ld[4]};
  return MKA_OK;
}

// ---------------------------------------------------------------- 8-bit cache
struct Kv {
  Kv8Args a;
  int Hq, G, bf16, window, sinks;
  float scale;
};
int check_kv8(const char* who, const mka_kv8_config* c, const mka_kv8_cache* cache, Kv* o) {
  if (!c) return fail(MKA_ERR_INVALID_ARG, "%s: cfg is NULL", who);
  if (c->batch < 1 || c->max_positions < 1) return fail(MKA_ERR_INVALID_ARG, "%s: batch and max_positions must be >= 1", who);
  const int e = check_heads(who, c->n_q_heads, c->n_kv_heads, c->d_head, c->attn_scale, &o->scale);
  if (e != MKA_OK) return e;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return fail(MKA_ERR_UNSUPPORTED, "%s: block must be 16, 32, 64 or 128", who);
  if (c->dtype != MKA_F32 && c->dtype != MKA_BF16) return fail(MKA_ERR_INVALID_ARG, "%s: dtype must be MKA_F32 or MKA_BF16", who);
  if (c->window < 0 || c->sinks < 0) return fail(MKA_ERR_INVALID_ARG, "%s: window and sinks must be >= 0", who);
  if (c->batch > 65535 || c->n_kv_heads > 32767 || c->max_positions > (1 << 28) ||
      (long long)c->n_q_heads * c->d_head > (1LL << 24) || (long long)c->batch * c->n_kv_heads > (1 << 20) ||
      (long long)c->batch * c->n_kv_heads * c->max_positions > 0x7fffffffLL - 128)
    return fail(MKA_ERR_UNSUPPORTED, "%s: batch, heads or max_positions too large", who);
  o->a = {nullptr, nullptr, nullptr, nullptr, c->batch, c->n_kv_heads, c->d_head, c->max_positions, c->block,
          (c->max_positions + c->block - 1) / c->block,
          c->block == 16 ? 4 : c->block == 32 ? 5 : c->block == 64 ? 6 : 7};
  o->Hq = c->n_q_heads;
  o->G = c->n_q_heads / c->n_kv_heads;
  o->bf16 = c->dtype == MKA_BF16;
  o->window = c->window >= c->max_positions ? 0 : c->window;
  o->sinks = o->window ? (c->sinks < c->max_positions ? c->sinks : c->max_positions) : 0;
  if (cache) {
    NEED(cache->k); NEED(cache->v);
    if (!cache->k_scale || !cache->v_scale || ((uintptr_t)cache->k_scale & 3) || ((uintptr_t)cache->v_scale & 3))
      return fail(MKA_ERR_INVALID_ARG, "%s: a scale pointer is NULL or misaligned", who);
    o->a.k = cache->k; o->a.v = cache->v; o->a.ks = cache->k_scale; o->a.vs = cache->v_scale;
  }
  return MKA_OK;
}
int check_positions(const char* who, const int32_t* p, const char* name, bool needed) {
  if (needed && !p) return fail(MKA_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if ((uintptr_t)p & 3) return fail(MKA_ERR_INVALID_ARG, "%s: %s is not aligned", who, name);
  return MKA_OK;
}
int check_rows(const char* who, const Kv& kv, int64_t row_stride, int64_t batch_stride, int32_t n) {
  const int per = kv.bf16 ? 8 : 4;  // elements of 16 bytes
  if (n < 1) return fail(MKA_ERR_INVALID_ARG, "%s: n must be >= 1", who);
  if (row_stride < (int64_t)kv.a.Hkv * kv.a.dh || row_stride % per || batch_stride < 0 || batch_stride % per)
    return fail(MKA_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes, rows at least n_kv_heads * d_head apart", who);
  if ((int64_t)n * kv.a.Hkv * (kv.a.dh / 16) > 0x7fffff00) return fail(MKA_ERR_UNSUPPORTED, "%s: n too large", who);
  return MKA_OK;
}
// Bytes of K's (V's) codes and of its scales.
size_t code_bytes(const Kv& kv) { return (size_t)kv.a.B * kv.a.Hkv * kv.a.Lmax * kv.a.dh; }
size_t scale_bytes(const Kv& kv) { return (size_t)kv.a.B * kv.a.Hkv * kv.a.nblk * 4; }
// Attention limits: grid dimensions and the flat count of 128-position tiles.
int check_kv8_attention(const char* who, const Kv& kv, int32_t n) {
  if (n < 1) return fail(MKA_ERR_INVALID_ARG, "%s: n must be >= 1", who);
  if ((long long)kv.G * n > (1 << 20) || (long long)kv.a.B * n * kv.Hq > (1LL << 30))
    return fail(MKA_ERR_UNSUPPORTED, "%s: too many query rows", who);
  const long long units = (long long)kv.a.Hkv * (((long long)kv.G * n + 7) / 8), tiles = (kv.a.Lmax + 127) / 128;
  if (units * tiles > 0x7fffffff || units * kv.a.B > 0x7fffffff)
    return fail(MKA_ERR_UNSUPPORTED, "%s: max_positions times query rows too large", who);
  return MKA_OK;
}
#define TRY(expr)                  \
  do {                             \
    const int t_ = (expr);         \
    if (t_ != MKA_OK) return t_;   \
  } while (0)

}  // namespace

extern "C" {

int mka_kv8_append(const mka_kv8_config* cfg, const mka_kv8_cache* cache, const void* k_new, const void* v_new,
                   int64_t row_stride, int64_t batch_stride, int32_t n, const int32_t* pos, const int32_t* count,
                   void* stream) {
  Kv kv;
  if (!cache) return fail(MKA_ERR_INVALID_ARG, "%s: cache is NULL", __func__);
  TRY(check_kv8(__func__, cfg, cache, &kv));
  TRY(check_rows(__func__, kv, row_stride, batch_stride, n));
  NEED(k_new); NEED(v_new);
  TRY(check_positions(__func__, pos, "pos", true));
  TRY(check_positions(__func__, count, "count", false));
  const size_t pb = (size_t)kv.a.B * 4, cb = code_bytes(kv), sb = scale_bytes(kv);
  TRY(check_apart(__func__, {{"pos", pos, pb, false}, {"count", count, pb, false}, {"cache.k", kv.a.k, cb, true},
                             {"cache.v", kv.a.v, cb, true}, {"cache.k_scale", kv.a.ks, sb, true},
                             {"cache.v_scale", kv.a.vs, sb, true}}));
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  CUDA_TRY(kv8_append(kv.a, k_new, v_new, kv.bf16, row_stride, batch_stride, n, pos, count, status, (cudaStream_t)stream));
  return MKA_OK;
}

int mka_kv8_read(const mka_kv8_config* cfg, const mka_kv8_cache* cache, const int32_t* first, const int32_t* rows,
                 int32_t n, void* k_out, void* v_out, int64_t row_stride, int64_t batch_stride, void* stream) {
  Kv kv;
  if (!cache) return fail(MKA_ERR_INVALID_ARG, "%s: cache is NULL", __func__);
  TRY(check_kv8(__func__, cfg, cache, &kv));
  TRY(check_rows(__func__, kv, row_stride, batch_stride, n));
  const int64_t width = (int64_t)kv.a.Hkv * kv.a.dh;
  if (cfg->batch > 1 && batch_stride < width) return fail(MKA_ERR_INVALID_ARG, "%s: the sequences' outputs are the same rows", __func__);
  NEED(k_out); NEED(v_out);
  TRY(check_positions(__func__, first, "first", false));
  TRY(check_positions(__func__, rows, "rows", false));
  const size_t wb = (size_t)width * (kv.bf16 ? 2 : 4);  // a row: K's and V's rows may lie in each other's gaps
  TRY(check_apart(__func__, {{"k_out", k_out, wb, true}, {"v_out", v_out, wb, true}}));
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  CUDA_TRY(kv8_read(kv.a, first, rows, n, k_out, v_out, kv.bf16, row_stride, batch_stride, status, (cudaStream_t)stream));
  return MKA_OK;
}

size_t mka_kv8_attention_workspace_size(const mka_kv8_config* cfg, int32_t n, int32_t with_weights) {
  Kv kv;
  size_t a, b;
  if (check_kv8(__func__, cfg, nullptr, &kv) != MKA_OK || check_kv8_attention(__func__, kv, n) != MKA_OK) return 0;
  return kv8_attention_scratch(kv.a, kv.G, n, with_weights, &a, &b);
}

int mka_kv8_attention(const mka_kv8_config* cfg, const mka_kv8_cache* cache, const void* q, int32_t n, const int32_t* lens,
                      void* out, float* weights, void* ws, size_t ws_bytes, void* stream) {
  Kv kv;
  if (!cache) return fail(MKA_ERR_INVALID_ARG, "%s: cache is NULL", __func__);
  TRY(check_kv8(__func__, cfg, cache, &kv));
  TRY(check_kv8_attention(__func__, kv, n));
  NEED(q); NEED(out); NEED(ws);
  TRY(check_positions(__func__, lens, "lens", true));
  if ((uintptr_t)weights & 3) return fail(MKA_ERR_INVALID_ARG, "%s: weights is not aligned", __func__);
  size_t stats, scores;
  const size_t need = kv8_attention_scratch(kv.a, kv.G, n, weights != nullptr, &stats, &scores);
  if (ws_bytes < need) return fail(MKA_ERR_WORKSPACE, "%s: ws holds %zu bytes, needs %zu", __func__, ws_bytes, need);
  const size_t rb = (size_t)kv.a.B * n * kv.Hq * kv.a.dh * (kv.bf16 ? 2 : 4);
  TRY(check_apart(__func__, {{"lens", lens, (size_t)kv.a.B * 4, false}, {"cache.k", kv.a.k, code_bytes(kv), false},
                             {"cache.v", kv.a.v, code_bytes(kv), false}, {"cache.k_scale", kv.a.ks, scale_bytes(kv), false},
                             {"cache.v_scale", kv.a.vs, scale_bytes(kv), false}, {"out", out, rb, true},
                             {"q", q == out ? nullptr : q, rb, false},  // (in place is safe: a unit's rows are its own)
                             {"weights", weights, (size_t)kv.a.B * kv.a.Hkv * kv.a.Lmax * 4, true}, {"ws", ws, need, true}}));
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  Kv8Attn a = {};
  a.c = kv.a;
  a.q = q; a.out = out; a.lens = lens; a.n = n; a.G = kv.G; a.window = kv.window; a.sinks = kv.sinks;
  a.sl2 = kv.scale * 1.4426950408889634f;
  a.part = (float*)ws;
  a.weights = weights;
  a.stats = (float*)((char*)ws + stats);
  a.scores = (float*)((char*)ws + scores);
  CUDA_TRY(kv8_attention(a, kv.bf16, status, (cudaStream_t)stream));
  return MKA_OK;
}

size_t mka_kv8_evict_workspace_size(const mka_kv8_config* cfg, int32_t keep) {
  Kv kv;
  if (check_kv8(__func__, cfg, nullptr, &kv) != MKA_OK || keep < 1) return 0;
  return 256;
}

int mka_kv8_evict(const mka_kv8_config* cfg, const mka_kv8_cache* cache, const int32_t* lens, const float* weights,
                  int32_t keep, int32_t first, int32_t recent, const mka_kv8_config* dst_cfg, const mka_kv8_cache* dst,
                  int32_t* dst_lens, float* dst_weights, int32_t* kept, void* ws, size_t ws_bytes, void* stream) {
  Kv s, d;
  if (!cache || !dst) return fail(MKA_ERR_INVALID_ARG, "%s: cache or dst is NULL", __func__);
  TRY(check_kv8(__func__, cfg, cache, &s));
  TRY(check_kv8(__func__, dst_cfg, dst, &d));
  if (d.a.B != s.a.B || d.a.Hkv != s.a.Hkv || d.a.dh != s.a.dh)
    return fail(MKA_ERR_INVALID_ARG, "%s: dst must have the batch, KV heads and head size of the cache", __func__);
  if (keep < 1 || first < 0 || recent < 0 || (int64_t)first + recent > keep)
    return fail(MKA_ERR_INVALID_ARG, "%s: keep must be >= 1 and first + recent within it", __func__);
  if (keep > d.a.Lmax) return fail(MKA_ERR_INVALID_ARG, "%s: keep exceeds the new cache", __func__);
  if (cache->k == dst->k || cache->v == dst->v || cache->k == dst->v || cache->v == dst->k || cache->k_scale == dst->k_scale || cache->v_scale == dst->v_scale ||
      (const void*)weights == dst_weights || (const void*)lens == dst_lens)
    return fail(MKA_ERR_INVALID_ARG, "%s: dst must be another cache", __func__);
  TRY(check_positions(__func__, lens, "lens", true));
  TRY(check_positions(__func__, dst_lens, "dst_lens", true));
  TRY(check_positions(__func__, kept, "kept", true));
  if (!weights || ((uintptr_t)weights & 3) || ((uintptr_t)dst_weights & 3))
    return fail(MKA_ERR_INVALID_ARG, "%s: weights is NULL or misaligned", __func__);
  NEED(ws);
  if (ws_bytes < mka_kv8_evict_workspace_size(cfg, keep)) return fail(MKA_ERR_WORKSPACE, "%s: ws is too small", __func__);
  const size_t heads = (size_t)s.a.B * s.a.Hkv, pb = (size_t)s.a.B * 4;
  TRY(check_apart(__func__, {{"lens", lens, pb, false}, {"weights", weights, heads * s.a.Lmax * 4, false},
                             {"cache.k", s.a.k, code_bytes(s), false}, {"cache.v", s.a.v, code_bytes(s), false},
                             {"cache.k_scale", s.a.ks, scale_bytes(s), false}, {"cache.v_scale", s.a.vs, scale_bytes(s), false},
                             {"dst.k", d.a.k, code_bytes(d), true}, {"dst.v", d.a.v, code_bytes(d), true},
                             {"dst.k_scale", d.a.ks, scale_bytes(d), true}, {"dst.v_scale", d.a.vs, scale_bytes(d), true},
                             {"dst_lens", dst_lens, pb, true}, {"dst_weights", dst_weights, heads * d.a.Lmax * 4, true},
                             {"kept", kept, heads * keep * 4, true}}));
  if (!device_status()) return fail(MKA_ERR_CUDA, "no CUDA device");
  CUDA_TRY(kv8_evict(s.a, lens, weights, keep, first, recent, d.a, dst_lens, dst_weights, kept, (cudaStream_t)stream));
  return MKA_OK;
}

int mka_window_attention(const mka_attn_config* cfg, const mka_attn_strides* strides, const void* q, const void* k,
                         const void* v, const int32_t* lens, void* out, float* lse, void* stream) {
  Win w;
  const int e = check_win(__func__, cfg, strides, &w);
  if (e != MKA_OK) return e;
  NEED(q); NEED(k); NEED(v); NEED(out); OPTIONAL(lse);
  if ((uintptr_t)lens & 3) return fail(MKA_ERR_INVALID_ARG, "%s: lens is not aligned", __func__);
  const int dq = w.Hq * w.dh, dkv = w.Hkv * w.dh;
  const long long rows = (long long)w.B * w.S;
  TRY(check_rows_apart(__func__, rows, {{"q", q, dq, w.ld.q, false}, {"k", k, dkv, w.ld.k, false}, {"v", v, dkv, w.ld.v, false},
                                        {"out", out, dq, w.ld.o, true}}));
  TRY(check_apart(__func__, {{"out", out, 2 * ((size_t)(rows - 1) * w.ld.o + dq), true}, {"lens", lens, (size_t)w.B * 4, false},
                             {"lse", lse, (size_t)w.B * w.Hq * w.Spad * 4, true}}));
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  AttnArgs a = {};
  a.q = q; a.q_ld = w.ld.q; a.q_bstride = (long long)w.S * w.ld.q;
  a.k = k; a.v = v; a.kv_ld = w.ld.k; a.kv_bstride = (long long)w.S * w.ld.k;
  a.v_ld = w.ld.v; a.v_bstride = (long long)w.S * w.ld.v;
  a.o = out; a.o_ld = w.ld.o; a.o_bstride = (long long)w.S * w.ld.o;
  a.B = w.B; a.S = w.S; a.Hq = w.Hq; a.Hkv = w.Hkv; a.dh = w.dh; a.scale = w.scale;
  a.lse = lse; a.lse_ld = w.Spad;
  a.windowed = true; a.window = w.window; a.sinks = w.sinks; a.lens = lens;
  CUDA_TRY(attention_prefill_tc(a, status, (cudaStream_t)stream));
  return MKA_OK;
}

size_t mka_window_attention_backward_workspace_size(const mka_attn_config* cfg) {
  Win w;
  if (check_win(__func__, cfg, nullptr, &w) != MKA_OK) return 0;
  return window_attention_backward_scratch(w.B, w.S, w.Hq, w.Hkv, w.dh, w.window, w.sinks, nullptr);
}

int mka_window_attention_backward(const mka_attn_config* cfg, const mka_attn_strides* strides, const void* q,
                                  const void* k, const void* v, const void* out, const float* lse, const void* dout,
                                  const int32_t* lens, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                  void* stream) {
  Win w;
  const int e = check_win(__func__, cfg, strides, &w);
  if (e != MKA_OK) return e;
  NEED(q); NEED(k); NEED(v); NEED(out); NEED(lse); NEED(dout); NEED(dq); NEED(dk); NEED(dv); NEED(ws);
  if ((uintptr_t)lens & 3) return fail(MKA_ERR_INVALID_ARG, "%s: lens is not aligned", __func__);
  size_t part = 0;
  const size_t need = window_attention_backward_scratch(w.B, w.S, w.Hq, w.Hkv, w.dh, w.window, w.sinks, &part);
  if (ws_bytes < need) return fail(MKA_ERR_WORKSPACE, "%s: ws holds %zu bytes, needs %zu", __func__, ws_bytes, need);
  const int nq = w.Hq * w.dh, nkv = w.Hkv * w.dh;
  const long long rows = (long long)w.B * w.S;
  TRY(check_rows_apart(__func__, rows, {{"q", q, nq, w.ld.q, false}, {"k", k, nkv, w.ld.k, false}, {"v", v, nkv, w.ld.v, false},
                                        {"out", out, nq, w.ld.o, false}, {"dout", dout, nq, w.ld.dout, false},
                                        {"dq", dq, nq, nq, true}, {"dk", dk, nkv, nkv, true}, {"dv", dv, nkv, nkv, true}}));
  TRY(check_apart(__func__, {{"lens", lens, (size_t)w.B * 4, false}, {"lse", lse, (size_t)w.B * w.Hq * w.Spad * 4, false},
                             {"dq", dq, 2 * (size_t)rows * nq, true}, {"dk", dk, 2 * (size_t)rows * nkv, true},
                             {"dv", dv, 2 * (size_t)rows * nkv, true}, {"ws", ws, need, true}}));
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  AttnBwdArgs a = {};
  a.q = q; a.k = k; a.v = v; a.dout = dout;
  a.lse = lse; a.lse_ld = w.Spad;
  a.B = w.B; a.S = w.S; a.Hq = w.Hq; a.Hkv = w.Hkv; a.dh = w.dh; a.scale = w.scale;
  a.window = w.window; a.sinks = w.sinks; a.lens = lens;
  a.dq16 = dq; a.dk16 = dk; a.dv16 = dv;
  a.sink_part = (float*)((char*)ws + part);
  CUDA_TRY(window_attention_backward_tc(a, w.ld, out, ws, status, (cudaStream_t)stream));
  return MKA_OK;
}

}  // extern "C"
