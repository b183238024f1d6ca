// C ABI of the bounded-memory attention operators: argument checks and launches.
// Declarations and the contract of every entry point are in include/mka.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

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

}  // namespace

extern "C" {

int mka_window_attention(const mka_attn_config* cfg, const mka_attn_strides* strides, const void* q, const void* k,
                         const void* v, const int32_t* lens, void* out, float* lse, void* stream) {
  Win w;
  const int e = check_win(__func__, cfg, strides, &w);
  if (e != MKA_OK) return e;
  NEED(q); NEED(k); NEED(v); NEED(out); OPTIONAL(lse);
  if ((uintptr_t)lens & 3) return fail(MKA_ERR_INVALID_ARG, "%s: lens is not aligned", __func__);
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
  int* status = device_status();
  if (!status) return fail(MKA_ERR_CUDA, "no CUDA device");
  AttnBwdArgs a = {};
  a.q = q; a.k = k; a.v = v; a.dout = dout;
  a.lse = lse; a.lse_ld = w.Spad;
  a.B = w.B; a.S = w.S; a.Hq = w.Hq; a.Hkv = w.Hkv; a.dh = w.dh; a.scale = w.scale;
  a.window = w.window; a.sinks = w.sinks; a.lens = lens;
  a.dq16 = dq; a.dk16 = dk; a.dv16 = dv;
  a.sink_part = (float*)((char*)ws + part);
  CUDA_TRY(window_attention_backward_tc(a, w.ld, out, (float*)ws, status, (cudaStream_t)stream));
  return MKA_OK;
}

}  // extern "C"
