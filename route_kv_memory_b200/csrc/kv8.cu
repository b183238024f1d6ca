// K/V cache held in 8 bits: append (quantise), read, attention of new tokens, eviction.
//
// Layout: codes [B][Hkv][Lmax][dh] e4m3, one float32 scale per (sequence, KV head, block of tokens)
// [B][Hkv][ceil(Lmax / block)]; a row's values are code * scale.  The scale of a block is the smallest
// power of two with max |value| <= 448 * scale (448: the largest e4m3 value).  A power of two costs the
// floating-point codes no precision, makes code * scale exact, and lets a block whose scale grows
// re-round its older codes without a second rounding error (only codes that fall below the smallest
// normal one change).
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "sm100.cuh"

namespace mka {

cudaError_t make_tmap_u8(CUtensorMap* map, const void* base, long long rows, int cols, int box_rows);

namespace kv8 {

constexpr float kQuietNaN = __builtin_nanf("");

// 2^x for x in [-126, 127].
__device__ __forceinline__ float pow2(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }
// The smallest x >= -120 with amax <= 448 * 2^x (amax finite, >= 0): amax = 1.f * 2^(E - 127) and
// 448 = 1.75 * 2^8, so x = E - 135, one more when the fraction exceeds .75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return max(-120, (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0));
}
__device__ __forceinline__ int exp_of(float p2) { return (int)(__float_as_uint(p2) >> 23) - 127; }

// x, an infinity as NaN.
__device__ __forceinline__ float finite_or_nan(float x) { return fmaf(x, 0.f, x); }
// Two values to e4m3 (a in the low byte): round to nearest even.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 codes (16 bits) to half2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t lo16) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)lo16));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t lo16) {
  const uint32_t h = e4m3x2_to_h2(lo16);
  return __half22float2(*(const __half2*)&h);
}

// 16 consecutive values as float (p 16-byte aligned).
template <typename T> __device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <> __device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = ((const float4*)p)[i];
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
template <> __device__ __forceinline__ void load16<bf16>(const bf16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = ((const uint4*)p)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
}
template <typename T> __device__ __forceinline__ void store16(T* p, const float (&x)[16]);
template <> __device__ __forceinline__ void store16<float>(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) ((float4*)p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <> __device__ __forceinline__ void store16<bf16>(bf16* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]);
      w[k] = *(const uint32_t*)&h;
    }
    ((uint4*)p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// 16 codes times a factor.
__device__ __forceinline__ void decode16(const uint4& c, float f, float (&x)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = e4m3x2_to_f2(w[k]), b = e4m3x2_to_f2(w[k] >> 16);
    x[4 * k] = a.x * f; x[4 * k + 1] = a.y * f; x[4 * k + 2] = b.x * f; x[4 * k + 3] = b.y * f;
  }
}
// 16 values times a power of two to codes; infinities become NaN.
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float inv) {
  uint32_t w[4];
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = fmaf(x[i], inv, x[i] * 0.f);
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = to_e4m3x2(y[4 * k], y[4 * k + 1]) | (to_e4m3x2(y[4 * k + 2], y[4 * k + 3]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// max |x| over the finite values.
__device__ __forceinline__ float amax16(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(finite_or_nan(x[i])));
  return m;
}
// (The append's and the read's traffic is rows in, codes out and in, values out: 2 x 4096, 28/4 heads,
// bf16: 50 MB in 14.4 us, two launches; a token a sequence: latency, 64 x 1: 7.6 us.)
// Codes of a scale 2^-d times as large: value * 2^d rounded once.  In half precision: a code times 2^d is
// exact there wherever it does not round to 0 (below 2^-10 it does, and a code of 4 significant bits that
// stays above is a multiple of 2^-14 at least), and the caller's scale keeps it within 448.
__device__ __forceinline__ uint4 rescale16(const uint4& c, int d) {
  d = min(max(d, -24), 18);
  const int d1 = min(max(d, -14), 15);
  const __half2 f1 = __float2half2_rn(pow2(d1)), f2 = __float2half2_rn(pow2(d - d1));
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = e4m3x2_to_h2(w[k] >> (16 * i));
      const __half2 y = __hmul2(__hmul2(*(const __half2*)&h, f1), f2);
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[i]) : "r"(*(const uint32_t*)&y));
    }
    w[k] = r[0] | (uint32_t)r[1] << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maximum over a block of NT threads (every thread gets it).
template <int NT>
__device__ __forceinline__ float block_max(float v, float* s) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = s[0];
#pragma unroll
  for (int i = 1; i < NT / 32; ++i) m = fmaxf(m, s[i]);
  return m;
}

// ============================================================================ append
// One block of threads per (touched token block, K or V and head, sequence).  The new rows of the token
// block stay in registers between the maximum and the codes, so each is read once.
constexpr int AP_THREADS = 128;

template <typename T, int DH, int CH>  // CH: 16-value chunks per thread, CH * AP_THREADS >= block * DH / 16
__global__ void __launch_bounds__(AP_THREADS) append_kernel(Kv8Args a, const T* kn, const T* vn, long long row_stride,
                                                            long long batch_stride, int n, const int* pos,
                                                            const int* count, int* status) {
  __shared__ float red[AP_THREADS / 32];
  constexpr int CPR = DH / 16;  // chunks per row
  const int b = blockIdx.z, kv = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
  allow_next_kernel();
  wait_previous_kernel();
  const int p = pos[b], c = count ? min(max(count[b], 0), n) : n;
  if (p < 0 || (long long)p + c > a.Lmax) {  // the whole sequence is left as it was
    if (threadIdx.x == 0) set_status(status, p < 0 ? kStatusBounds : kStatusCapacity);
    return;
  }
  const int tb = (p >> a.lb) + blockIdx.x, t0 = tb * a.block;
  const int lo = max(p, t0), hi = min(p + c, t0 + a.block);  // new rows of this token block
  if (lo >= hi) return;
  uint8_t* codes = (uint8_t*)(kv ? a.v : a.k) + ((size_t)b * a.Hkv + g) * a.Lmax * DH;
  float* scale = (kv ? a.vs : a.ks) + ((size_t)b * a.Hkv + g) * a.nblk + tb;
  const T* x = (kv ? vn : kn) + (size_t)b * batch_stride + (size_t)g * DH;
  const int nch = (hi - lo) * CPR;
  float v[CH][16], m = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int ch = i * AP_THREADS + threadIdx.x;
    if (ch < nch) {
      load16<T>(x + (size_t)(lo - p + ch / CPR) * row_stride + ch % CPR * 16, v[i]);
      m = fmaxf(m, amax16(v[i]));
    }
  }
  const float old = lo > t0 ? *scale : 0.f;  // the scale of the rows that the block already holds
  m = block_max<AP_THREADS>(m, red);         // (also: every thread has read the old scale)
  int e = scale_exp(m);
  if (lo > t0) e = max(e, exp_of(old));
  const float inv = pow2(-e);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int ch = i * AP_THREADS + threadIdx.x;
    if (ch < nch) *(uint4*)(codes + (size_t)(lo + ch / CPR) * DH + ch % CPR * 16) = encode16(v[i], inv);
  }
  if (lo > t0 && e != exp_of(old)) {
    for (int ch = threadIdx.x; ch < (lo - t0) * CPR; ch += AP_THREADS) {
      uint4* at = (uint4*)(codes + (size_t)(t0 + ch / CPR) * DH + ch % CPR * 16);
      *at = rescale16(*at, exp_of(old) - e);
    }
  }
  if (threadIdx.x == 0) *scale = pow2(e);
}

// ============================================================================ read
// Rows [first[b], first[b] + rows[b]) of sequence b to rows 0.. of the outputs; a block takes one head of K
// or V, a thread NC chunks of 16 codes, 256 apart, with all their loads in flight.
template <typename T, int DH, int NC>
__global__ void __launch_bounds__(256) read_kernel(Kv8Args a, const int* first, const int* rows, int n, T* k_out,
                                                   T* v_out, long long row_stride, long long batch_stride, int* status) {
  constexpr int CPR = DH / 16;
  const int b = blockIdx.z, kv = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
  allow_next_kernel();
  wait_previous_kernel();
  const int f = first ? first[b] : 0, r = rows ? min(max(rows[b], 0), n) : n;
  if (f < 0 || (long long)f + r > a.Lmax) {
    if (threadIdx.x == 0) set_status(status, kStatusBounds);
    return;
  }
  const size_t hd = (size_t)b * a.Hkv + g;
  const uint8_t* codes = (const uint8_t*)(kv ? a.v : a.k) + (hd * a.Lmax + f) * DH;
  const float* sc = (kv ? a.vs : a.ks) + hd * a.nblk;
  T* out = (kv ? v_out : k_out) + (size_t)b * batch_stride + g * DH;
  const int at = blockIdx.x * (256 * NC) + threadIdx.x, ch = at % CPR;
  uint4 v[NC];
  float s[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int row = (at + i * 256) / CPR;
    if (row < r) {
      v[i] = *(const uint4*)(codes + (size_t)row * DH + ch * 16);
      s[i] = sc[(f + row) >> a.lb];
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int row = (at + i * 256) / CPR;
    if (row < r) {
      float y[16];
      decode16(v[i], s[i], y);
      store16<T>(out + (size_t)row * row_stride + ch * 16, y);
    }
  }
}

// ============================================================================ attention
// A unit is (sequence b, KV head g, group of 8 NT query rows); a query row is (new token i, query head of
// g), row r = i * G + head.  Everything is computed transposed: S^T = K Q^T with 16 cached tokens as the
// rows of a m16n8k16 product and 8 query rows as its columns, O^T = V^T P^T with 16 channels as the rows:
// with a handful of query rows per KV head this wastes half as much of the products as 16-row query
// tiles would.  A contraction index may be permuted freely, and the channel order of O^T too, so the 16
// consecutive bytes that a lane loads of a token's row serve as its fragments without any transposition
// (K: bytes 4w..4w+3 of its pieces are k-step w; V: byte pairs of two tokens, joined by prmt).
// e4m3 to half is exact; q enters as half after a power-of-two scaling of its row (SPLIT, float32 q: as
// high and low halves); P as half, 2^HELD times its size relative to the row's running reference, so that
// it is off by 2^-11 of itself at most down to 2^-23 of the reference, and by 2^-34 of the reference below
// that: half's numbers end at 2^-24, and weights left out there would still be in the softmax's sum.  SPLIT
// carries the rest of that rounding as a second half 2^LOW as large, against codes 2^-LOW as large (multiples
// of 2^-20: exact): off by 2^-22 of itself, or 2^-45 of the reference.
//
// Every warp streams its own 32 tokens of each 128-token tile through its own two stages of shared
// memory, filled by TMA (K and V, 32 rows each) with the 128-byte (d_head 64: 64-byte) swizzle: no
// barrier across warps in the loop, 16 KB per warp in flight.  The token order inside 16 rows
// (slot_token) is chosen so that both kinds of fragment loads are free of bank conflicts.
//
// Work: the 128-token tiles that a unit's rows see, over all units in order, are cut into ranges of equal
// length (give or take one tile), one per CTA, so ragged batches stay balanced; a unit that falls into several ranges leaves partial
// results (slot = CTA + unit, which increases along the ranges and never repeats) for merge_kernel.
//
// Bound by HBM, of which the 36 MB in flight keep 88% busy from the first copy (2.9 us after the start:
// lens, the split, the queries) to the last: 1 x 131072, 28/4 heads, d_head 128, one new token: 134 MB,
// 28 us and the merge 4 us more; 16 sequences of up to 32768, 32/8 heads, 4 new tokens: 571 MB on
// average, 107 us.
constexpr int AT_THREADS = 128;
constexpr int TILE = 128;      // tokens per CTA step, 32 per warp
constexpr int STAGES = 2;      // per warp
// log2: the reference moves when it is exceeded by more than LAZY; P, held 2^HELD as large, stays below 2^15,
// and the low half below 2^15 too (half a step of the high one, 2^4, times 2^LOW).  LAZY + HELD = 15 splits
// half's range between rare moves and small weights: 8 + 7 / 6 + 9 / 4 + 11 take 106.3 / 106.8 / 108.3 us for
// 16 sequences of up to 32768 with 4 new tokens, 32.0 each for 1 x 131072.
constexpr float LAZY = 6.f;
constexpr int HELD = 9, LOW = 11;

struct Tiles {  // the 128-token tiles of a unit: tile i at i < nsk ? i : lo + i - nsk
  int len, lo, nsk, n;
  __device__ __forceinline__ int tile(int i) const { return i < nsk ? i : lo + i - nsk; }
};
__device__ __forceinline__ Tiles unit_tiles(const Kv8Attn& a, int b) {
  Tiles t;
  t.len = min(max(a.lens[b], 0), a.c.Lmax);
  const int p0 = max(t.len - a.n, 0);  // the first query that has a position
  t.lo = a.window ? max(0, p0 - a.window + 1) / TILE : 0;
  t.nsk = min((a.sinks + TILE - 1) / TILE, t.lo);
  t.n = t.len > 0 ? t.nsk + (t.len - 1) / TILE - t.lo + 1 : 0;
  return t;
}
// a / b of non-negative numbers; 64-bit divisions, a microsecond in a chain of them, only where they are needed.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
struct Split {  // `total` tiles over `grid` CTAs: the first `more` of them take one tile more than the others
  long long base, more;
  __device__ __forceinline__ Split(long long total, int grid) : base(quotient(total, grid)), more(total - base * grid) {}
  __device__ __forceinline__ long long start(long long cta) const { return cta * base + min(cta, more); }
  __device__ __forceinline__ int cta_of(long long tile) const {
    return (int)(tile < more * (base + 1) ? quotient(tile, base + 1) : more + quotient(tile - more * (base + 1), base));
  }
};
__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ uint32_t times_h2(uint32_t u, float f) {  // both halves times f (exact where f is a power of two)
  const __half2 h = __hmul2(*(const __half2*)&u, __float2half2_rn(f));
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t u) { return __half22float2(*(const __half2*)&u); }

// Token (0..7) of row x (0..7) of an 8-row half of a S^T tile = contraction index x of O^T.  d_head 128
// (128-byte rows, 16-byte chunk c of row t at chunk c ^ t): rows x and x ^ 1 differ in bit 2, so that
// their K chunks 0-3 (4-7) land in different halves, and rows 0, 2, 4, 6 (1, 3, 5, 7) differ in bits 1-2,
// so that V chunks 2y and 2y + 1 of the four lanes' tokens never meet.
template <int DH> __device__ __forceinline__ int slot_token(int x) {
  return DH == 128 ? ((x >> 2) & 1) | (x & 2) | (((x ^ (x >> 2)) & 1) << 2) : x;
}
// Byte offset of byte `at` of row t in a swizzled tile.
template <int DH> __device__ __forceinline__ int swizzled(int t, int at) {
  return DH == 128 ? t * 128 + (at ^ ((t & 7) << 4)) : t * 64 + (at ^ (((t >> 1) & 3) << 4));
}

template <int DH> struct AtCfg {
  static constexpr int HALF = 32 * DH;            // 32 rows of K (or V)
  static constexpr int WARP = STAGES * 2 * HALF;  // a warp's stages: K, V
  static constexpr int SMEM = 4 * WARP + 1024;
};

// O of a row from the products' sum: / sum, * 2^(U - L), the references of the products and of the sum, U HELD low.
// In two factors: V's scales reach down to 2^-120, and 2^x is 0 below 2^-126.
struct Norm {
  float a, b;
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};
__device__ __forceinline__ Norm row_norm(float L, float U, float sum) {
  return {sum == 0.f ? 0.f : 1.f / (1 << HELD) / sum, sum == 0.f ? 0.f : sm100::ex2(U + (float)HELD - L)};  // nothing seen: 0
}

// NT: groups of 8 query rows; SPLIT: float32 queries and outputs; WT: raw scores go to a.scores.
template <typename T, int DH, int NT, bool WT>
__global__ void __launch_bounds__(AT_THREADS, DH == 128 && NT == 2 ? 2 : 3)
    attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Kv8Attn a, int* status) {
  using namespace sm100;
  using C = AtCfg<DH>;
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int KW = DH / 16;      // 32-bit words of a K row per lane = k-steps of S^T
  constexpr int MT = DH / 16;      // 16-channel tiles of O^T
  constexpr int VW = DH / 32;      // 32-bit words of a V row per lane
  constexpr int RT = 8 * NT;
  constexpr int OLD = DH + 4;      // row stride of the warps' O in shared memory
  static_assert(RT * OLD * 4 <= C::WARP, "a warp's O fits its stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t bars[4][STAGES];
  __shared__ float sStat[4][RT][3];  // ml, l, mu of each warp
  __shared__ long long sScan[AT_THREADS / 32];
  __shared__ int sStart[2];
  __shared__ Tiles sTiles;
  __shared__ int sAbort;
  volatile int* abort = &sAbort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, c4 = lane & 3;
  const int R = a.G * a.n, nrg = (R + RT - 1) / RT, upb = a.c.Hkv * nrg;  // units per sequence
  uint8_t* mine = smem + warp * C::WARP;
  uint64_t* full = bars[warp];

  if (threadIdx.x == 0) {
    sAbort = 0;
    for (int i = 0; i < 4; ++i)
      for (int k = 0; k < STAGES; ++k) mbar_init(&bars[i][k], 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  wait_previous_kernel();
  allow_next_kernel();  // (not before: merge_kernel reads lens ahead of its own wait)
  // this CTA's range of tiles [w0, w1) and the sequence that w0 falls into
  long long total;
  Split split(0, 1);
  {
    const int per = (a.c.B + AT_THREADS - 1) / AT_THREADS, b0 = min(threadIdx.x * per, a.c.B), b1 = min(b0 + per, a.c.B);
    long long own = 0;
    for (int b = b0; b < b1; ++b) own += (long long)unit_tiles(a, b).n * upb;
    long long inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sScan[warp] = inc;
    __syncthreads();
    long long before = inc - own;
    total = 0;
    for (int i = 0; i < AT_THREADS / 32; ++i) {
      if (i < warp) before += sScan[i];
      total += sScan[i];
    }
    split = Split(total, gridDim.x);
    const long long w0 = split.start(blockIdx.x);
    if (w0 >= before && w0 < before + own) {  // one thread at most
      long long left = w0 - before;
      int b = b0;
      for (;; ++b) {
        const Tiles x = unit_tiles(a, b);
        const long long t = (long long)x.n * upb;
        if (left < t) {
          sTiles = x;
          break;
        }
        left -= t;
      }
      sStart[0] = b;
      sStart[1] = (int)left;  // tiles of sequence b before w0
    }
    __syncthreads();
  }
  int todo = (int)(split.start(blockIdx.x + 1) - split.start(blockIdx.x)), b = sStart[0];
  if (todo == 0) return;
  Tiles ts = sTiles;
  int u = sStart[1] / ts.n, first = sStart[1] % ts.n;  // unit within the sequence, its first tile here
  int kvit = 0;  // tiles this warp has taken from its stages
  const uint64_t pol = policy_evict_first();  // the cache is read once

  // lane constants: offsets of its pieces in a 32-row stage
  int koff[DH / 64], voff[2];
#pragma unroll
  for (int q = 0; q < DH / 64; ++q) koff[q] = swizzled<DH>(slot_token<DH>(g8), q * 64 + c4 * 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) voff[i] = swizzled<DH>(slot_token<DH>(2 * c4 + i), g8 * (DH / 8));

  while (todo > 0) {
    const int cnt = min(todo, ts.n - first);
    const int g = u / nrg, rg = u % nrg;
    const size_t hd = (size_t)b * a.c.Hkv + g;
    const int row0 = (int)(hd * a.c.Lmax);
    const float* ksc = a.c.ks + hd * a.c.nblk;
    const float* vsc = a.c.vs + hd * a.c.nblk;
    auto fetch = [&](int it, int st) {  // lane 0: this warp's rows of the segment's tile `it` into stage st
      const int y = row0 + ts.tile(first + it) * TILE + warp * 32;
      mbar_expect_tx(&full[st], 2 * C::HALF);
      tma_load_2d_hint(mine + st * 2 * C::HALF, &tmK, &full[st], 0, y, pol);
      tma_load_2d_hint(mine + st * 2 * C::HALF + C::HALF, &tmV, &full[st], 0, y, pol);
    };
    // the queries' loads go first: behind the first tiles they would wait for all of those (4 us at
    // 131072 tokens, 36 MB in flight)
    float qx[NT][KW / 4][16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = min(rg * RT + t * 8 + g8, R - 1);
      const T* qr = (const T*)a.q + ((size_t)b * a.n + r / a.G) * (size_t)(a.c.Hkv * a.G * DH) +
                    (size_t)(g * a.G + r % a.G) * DH;
#pragma unroll
      for (int q = 0; q < KW / 4; ++q) load16<T>(qr + q * 64 + c4 * 16, qx[t][q]);
    }
    if (lane == 0) {
      fence_proxy_async();  // (the stages held this warp's O of the segment before)
      for (int i = 0; i < STAGES && i < cnt; ++i) fetch(i, (kvit + i) % STAGES);
    }

    // Q^T fragments of row g8 of each group: k-step w holds the channels of bytes 4w..4w+3 of the
    // lane's K pieces; the row is scaled by a power of two to a maximum in [2^7, 2^8)
    uint32_t qf[NT][KW][2], ql[SPLIT ? NT : 1][SPLIT ? KW : 1][2];
    float rf[NT][2];       // score factor of the rows of this lane's accumulators (2 c4 and 2 c4 + 1)
    int qpos[NT][2];       // their positions; -1: not a row
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bool in = rg * RT + t * 8 + g8 < R;
      float(&x)[KW / 4][16] = qx[t];
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < KW / 4; ++q) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (!in) x[q][i] = 0.f;
          m = fmaxf(m, fabsf(x[q][i]));
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = min(max((int)(__float_as_uint(m) >> 23) - 127 - 7, -119), 119);
      const float down = pow2(-e);
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float y0 = x[w >> 2][(w & 3) * 4 + 2 * i] * down, y1 = x[w >> 2][(w & 3) * 4 + 2 * i + 1] * down;
          qf[t][w][i] = pack_h2(y0, y1);
          if constexpr (SPLIT) {
            const float2 h = unpack_h2(qf[t][w][i]);
            ql[t][w][i] = pack_h2(y0 - h.x, y1 - h.y);
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rf[t][i] = pow2(__shfl_sync(0xffffffffu, e, (2 * c4 + i) * 4)) * a.sl2;
        const int rr = rg * RT + t * 8 + 2 * c4 + i;
        qpos[t][i] = rr < R ? ts.len - a.n + rr / a.G : -1;
      }
    }
    const int p_lo = ts.len - a.n + rg * RT / a.G, p_hi = ts.len - a.n + (min(R, (rg + 1) * RT) - 1) / a.G;

    float o[MT][NT][4], l[NT][2], ml[NT][2], mu[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] = 0.f;
        ml[t][i] = mu[t][i] = -INFINITY;
      }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][t][i] = 0.f;
    auto sees = [&](int j, int p) { return j <= p && (!a.window || j > p - a.window || j < a.sinks); };

    float nks[2], nvs[2];  // the scales of the next tile's two halves, loaded a tile ahead
    auto load_scales = [&](int it) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tb = min((ts.tile(first + it) * TILE + warp * 32 + 16 * h) >> a.c.lb, a.c.nblk - 1);
        nks[h] = ksc[tb];
        nvs[h] = vsc[tb];
      }
    };
    load_scales(0);
    for (int it = 0; it < cnt; ++it, ++kvit) {
      const int st = kvit % STAGES, j0 = ts.tile(first + it) * TILE + warp * 32;
      const uint8_t* sk = mine + st * 2 * C::HALF;
      const uint8_t* sv = sk + C::HALF;
      const float kf[2] = {nks[0], nks[1]}, ev[2] = {(float)exp_of(nvs[0]), (float)exp_of(nvs[1])};
      if (it + 1 < cnt) load_scales(it + 1);
      if (!mbar_wait_warp(&full[st], (kvit / STAGES) & 1, abort, status)) break;
      // S^T of 32 tokens
      float s[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[h][t][i] = 0.f;
#pragma unroll
        for (int q = 0; q < DH / 64; ++q) {
          const uint4 x0 = *(const uint4*)(sk + h * 16 * DH + koff[q]), x1 = *(const uint4*)(sk + (h * 16 + 8) * DH + koff[q]);
          const uint32_t y0[4] = {x0.x, x0.y, x0.z, x0.w}, y1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_h2(y0[w]), a1 = e4m3x2_to_h2(y1[w]), a2 = e4m3x2_to_h2(y0[w] >> 16),
                           a3 = e4m3x2_to_h2(y1[w] >> 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816(s[h][t], a0, a1, a2, a3, qf[t][q * 4 + w][0], qf[t][q * 4 + w][1]);
              if constexpr (SPLIT) mma16816(s[h][t], a0, a1, a2, a3, ql[t][q * 4 + w][0], ql[t][q * 4 + w][1]);
            }
          }
        }
      }

      // hidden scores -inf; s[h][t][i]: token j0 + 16 h + 8 (i / 2) + slot_token(g8), row 2 c4 + i % 2
      const bool edge = j0 + 31 > p_lo || (a.window && j0 <= p_hi - a.window && j0 + 31 >= a.sinks);  // warp-uniform
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!sees(j0 + 16 * h + 8 * (i >> 1) + slot_token<DH>(g8), qpos[t][i & 1])) s[h][t][i] = -INFINITY;
      }
      if constexpr (WT) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // the two rows of a token; a token's rows are padded to whole groups
              const int j = j0 + 16 * h + 8 * i + slot_token<DH>(g8);
              float2 x = make_float2(s[h][t][2 * i] * (kf[h] * rf[t][0]), s[h][t][2 * i + 1] * (kf[h] * rf[t][1]));
              if (edge) {  // (a hidden score times a factor of 0 would be NaN)
                if (s[h][t][2 * i] == -INFINITY) x.x = -INFINITY;
                if (s[h][t][2 * i + 1] == -INFINITY) x.y = -INFINITY;
              }
              if (j < ts.len) *(float2*)(a.scores + (hd * a.c.Lmax + j) * (nrg * RT) + rg * RT + t * 8 + 2 * c4) = x;
            }
      }
      // scores in log2 units are s * f; two references per row, for the sum (ml) and, with the exponent
      // ev of V's block scale added and HELD taken off, for the products with V's codes (mu)
      bool over = false;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            over |= fmaxf(s[h][t][k], s[h][t][k + 2]) * (kf[h] * rf[t][k]) > fminf(ml[t][k], mu[t][k] + HELD - ev[h]) + LAZY;
      if (__any_sync(0xffffffffu, over)) {  // move the references to the tile's maxima
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = -INFINITY, y = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float z = fmaxf(s[h][t][k], s[h][t][k + 2]), v = z == -INFINITY ? z : z * (kf[h] * rf[t][k]);
              x = fmaxf(x, v);
              y = fmaxf(y, v + (ev[h] - HELD));
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            }
            if (x > ml[t][k]) {
              l[t][k] *= ex2(ml[t][k] - x);
              ml[t][k] = x;
            }
            if (y > mu[t][k]) {
              const float f = ex2(mu[t][k] - y);
              mu[t][k] = y;
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                o[m][t][k] *= f;
                o[m][t][k + 2] *= f;
              }
            }
          }
      }
      // P^T: the fragments of S^T transposed into those of a B operand
      uint32_t pf[2][NT][2], pl[2][SPLIT ? NT : 1][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float x = s[h][t][2 * i + k], f = kf[h] * rf[t][k];
              const bool hid = edge && x == -INFINITY;
              y[k] = hid ? 0.f : ex2(fmaf(x, f, ev[h] - mu[t][k]));
              l[t][k] += hid ? 0.f : ex2(fmaf(x, f, -ml[t][k]));
            }
            const uint32_t hi = pack_h2(y[0], y[1]);
            pf[h][t][i] = transpose8x8(hi);
            if constexpr (SPLIT) {
              const float2 f = unpack_h2(hi);
              pl[h][t][i] = transpose8x8(pack_h2((y[0] - f.x) * (1 << LOW), (y[1] - f.y) * (1 << LOW)));
            }
          }
      // O^T += V^T P^T; channel tile m holds the channels 2m and 2m + 1 of each lane's piece; piece i is
      // of contraction index 2 c4 + i % 2 + 8 (i / 2)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t vr[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* p = sv + (h * 16 + 8 * (i >> 1)) * DH + voff[i & 1];
          if constexpr (DH == 128) {
            const uint4 x = *(const uint4*)p;
            vr[i][0] = x.x; vr[i][1] = x.y; vr[i][2] = x.z; vr[i][3] = x.w;
          } else {
            const uint2 x = *(const uint2*)p;
            vr[i][0] = x.x; vr[i][1] = x.y;
          }
        }
        if (edge) {
          // a hidden token's P is 0, but 0 * NaN is not: NaN codes are cleared, and the rows that do see
          // such a token get their NaN directly
          uint32_t nan[4], any = 0;  // bit d: channel d of this lane's piece i is NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            nan[i] = 0;
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (((vr[i][w] >> (8 * k)) & 0x7f) == 0x7f) {
                  nan[i] |= 1u << (4 * w + k);
                  vr[i][w] &= ~(0xffu << (8 * k));
                }
            any |= nan[i];
          }
          if (__any_sync(0xffffffffu, any != 0)) {
            for (int src = 0; src < 4; ++src)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t bits = __shfl_sync(0xffffffffu, nan[i], (lane & ~3) | src);
                const int j = j0 + 16 * h + 8 * (i >> 1) + slot_token<DH>(2 * src + (i & 1));
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int k = 0; k < 2; ++k)
                    if (bits && sees(j, qpos[t][k]))
#pragma unroll
                      for (int m = 0; m < MT; ++m) {
                        if ((bits >> (2 * m)) & 1) o[m][t][k] = kQuietNaN;
                        if ((bits >> (2 * m + 1)) & 1) o[m][t][k + 2] = kQuietNaN;
                      }
              }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t sel = (m & 1) ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(vr[0][m >> 1], vr[1][m >> 1], sel);
          const uint32_t y = __byte_perm(vr[2][m >> 1], vr[3][m >> 1], sel);
          const uint32_t a0 = e4m3x2_to_h2(x), a1 = e4m3x2_to_h2(x >> 16), a2 = e4m3x2_to_h2(y), a3 = e4m3x2_to_h2(y >> 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(o[m][t], a0, a1, a2, a3, pf[h][t][0], pf[h][t][1]);
          if constexpr (SPLIT) {
            const uint32_t l0 = times_h2(a0, pow2(-LOW)), l1 = times_h2(a1, pow2(-LOW)), l2 = times_h2(a2, pow2(-LOW)),
                           l3 = times_h2(a3, pow2(-LOW));
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(o[m][t], l0, l1, l2, l3, pl[h][t][0], pl[h][t][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && it + STAGES < cnt) fetch(it + STAGES, st);
    }

    // join the four warps, each one's O in its own stages (none of its copies is in flight)
    float* so = (float*)mine;
    if (!__any_sync(0xffffffffu, *abort)) {  // (one answer for the warp: shuffles follow)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = l[t][i];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
          const int r = t * 8 + 2 * c4 + i;
          if (g8 == 0) {
            sStat[warp][r][0] = ml[t][i];
            sStat[warp][r][1] = x;
            sStat[warp][r][2] = mu[t][i];
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
            *(float2*)&so[r * OLD + g8 * (DH / 8) + 2 * m] = make_float2(o[m][t][i], o[m][t][i + 2]);
        }
    }
    __syncthreads();  // (no wait follows in the segment: every thread sees the same abort)
    if (*abort) break;
    const bool whole = first == 0 && cnt == ts.n;
    const size_t slot = (size_t)blockIdx.x + (size_t)b * upb + u;
    for (int at = threadIdx.x; at < RT * (DH / 4); at += AT_THREADS) {
      const int r = at / (DH / 4), d = at % (DH / 4) * 4, row = rg * RT + r;
      if (row >= R) continue;
      float L = -INFINITY, U = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        L = fmaxf(L, sStat[w][r][0]);
        U = fmaxf(U, sStat[w][r][2]);
      }
      float sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // (a warp that saw nothing holds zeros, or the NaN of a NaN score: added as it is)
        sum += sStat[w][r][0] == -INFINITY ? sStat[w][r][1] : sStat[w][r][1] * ex2(sStat[w][r][0] - L);
        const float4 y = *(const float4*)((const float*)(smem + w * C::WARP) + r * OLD + d);
        const float f = sStat[w][r][2] == -INFINITY ? 1.f : ex2(sStat[w][r][2] - U);
        x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
      }
      if (whole) {
        const Norm f = row_norm(L, U, sum);
        T* out = (T*)a.out + ((size_t)b * a.n + row / a.G) * (size_t)(a.c.Hkv * a.G * DH) +
                 (size_t)(g * a.G + row % a.G) * DH + d;
        out[0] = from_f<T>(f(x.x)); out[1] = from_f<T>(f(x.y)); out[2] = from_f<T>(f(x.z)); out[3] = from_f<T>(f(x.w));
        if (WT && d == 0) *(float2*)(a.stats + 2 * (hd * R + row)) = make_float2(L, sum);
      } else {
        float* rec = a.part + (slot * RT + r) * (DH + 4);
        *(float4*)(rec + 4 + d) = x;
        if (d == 0) *(float4*)rec = make_float4(L, sum, U, 0.f);
      }
    }
    __syncthreads();
    todo -= cnt;
    first = 0;
    if (todo > 0 && ++u == upb) {
      u = 0;
      do ts = unit_tiles(a, ++b);
      while (ts.n == 0);
    }
  }
  if (threadIdx.x == 0) linger_after_abort(abort);  // a wait ran out: this CTA's copies land first
}

// The ranges' records of one unit's query rows.
struct Records {
  const float* p;  // the first range's record of row 0 of the row group: maximum, sum, reference of O, -, O
  size_t step;     // to the next range's
  int n;           // ranges; 1: the unit's CTA wrote its rows (and stats) itself
};
__device__ __forceinline__ Records unit_records(const Kv8Attn& a, int RT, int DH, int grid, long long before,
                                                long long total, int b, int u, int upb, int tiles) {
  const Split split(total, grid);
  const long long start = before + (long long)u * tiles;
  const int c0 = split.cta_of(start);
  return {a.part + ((size_t)b * upb + u + c0) * RT * (DH + 4), (size_t)RT * (DH + 4),
          split.cta_of(start + tiles - 1) - c0 + 1};
}

// weights[b][g][j] += sum over the query rows of KV head g of their softmax weight of token j, from the raw
// scores (log2 units) and each row's maximum and sum, which every CTA joins from the records for itself.
// A block takes WG_TILES of the unit's tiles, a thread WG_TOKENS tokens 256 apart.
constexpr int WG_THREADS = 256;  // = MG_THREADS
constexpr int WG_TOKENS = 4, WG_TILES = WG_TOKENS * WG_THREADS / TILE;
__device__ __forceinline__ void add_weights(const Kv8Attn& a, int RT, int DH, int grid, long long before, long long total,
                                            int block, int g, int b, const Tiles& ts) {
  using sm100::ex2;
  constexpr int ROWS = 64;  // rows whose normalisers are in shared memory at a time
  __shared__ __align__(16) float lse[ROWS];  // maximum + log2(sum)
  const int R = a.G * a.n, nrg = (R + RT - 1) / RT, upb = a.c.Hkv * nrg, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t hd = (size_t)b * a.c.Hkv + g;
  int j[WG_TOKENS];  // positions; -1: none
  float w[WG_TOKENS] = {};
#pragma unroll
  for (int k = 0; k < WG_TOKENS; ++k) {
    const int i = WG_TILES * block + 2 * k + (threadIdx.x >> 7), p = i < ts.n ? ts.tile(i) * TILE + (threadIdx.x & 127) : -1;
    j[k] = p < ts.len ? p : -1;
  }
  for (int r0 = 0; r0 < R; r0 += ROWS) {
    const int m = min(ROWS, (R - r0 + 3) & ~3);  // (rows behind R: the padding of the scores, weighed 0)
    __syncthreads();
    for (int r = warp; r < m; r += WG_THREADS / 32) {
      const int row = r0 + r, rg = row / RT;
      float L = -INFINITY, sum = 0.f;
      if (row < R) {
        const Records rec = unit_records(a, RT, DH, grid, before, total, b, g * nrg + rg, upb, ts.n);
        if (rec.n == 1) {
          if (lane == 0) {
            const float2 x = *(const float2*)(a.stats + 2 * (hd * R + row));
            L = x.x;
            sum = x.y;
          }
        } else {
          for (int c = lane; c < rec.n; c += 32) {
            const float2 h = *(const float2*)(rec.p + c * rec.step + (size_t)(row % RT) * (DH + 4));
            const float nl = fmaxf(L, h.x);
            sum = (L == -INFINITY ? sum : sum * ex2(L - nl)) + (h.x == -INFINITY ? h.y : h.y * ex2(h.x - nl));
            L = nl;
          }
        }
        const float all = warp_max(L);
        sum = warp_sum(L == -INFINITY ? sum : sum * ex2(L - all));
        L = all;
      }
      // (a row that sees nothing: every score -inf, weighed 0 by any finite normaliser; a row whose normaliser is NaN:
      // one so low that what the row sees is weighed infinitely, NaN below, and a hidden position still 0)
      if (lane == 0) {
        const float norm = L == -INFINITY && sum == 0.f ? 0.f : L + log2f(sum);
        lse[r] = row >= R ? INFINITY : norm != norm ? -3e38f : norm;
      }
    }
    __syncthreads();
    for (int r = 0; r < m; r += 4) {
      const float4 x = *(const float4*)(lse + r);
#pragma unroll
      for (int k = 0; k < WG_TOKENS; ++k)
        if (j[k] >= 0) {
          const float4 y = *(const float4*)(a.scores + (hd * a.c.Lmax + j[k]) * (size_t)(nrg * RT) + r0 + r);
          w[k] += ex2(y.x - x.x) + ex2(y.y - x.y) + ex2(y.z - x.z) + ex2(y.w - x.w);
        }
    }
  }
#pragma unroll
  for (int k = 0; k < WG_TOKENS; ++k)
    if (j[k] >= 0) a.weights[hd * a.c.Lmax + j[k]] += finite_or_nan(w[k]);
}

// Joins the partial results of the query rows; a unit without tiles gives 0.  WPR warps per row: 8 (a CTA
// per row) where a unit lies over many CTAs' ranges, 1 (8 rows a CTA) where it lies over a few.  WT: the
// blocks behind the rows' add up the weights.
constexpr int MG_THREADS = 256;
constexpr int MG_MOST = 1024;  // CTAs of the attention at most
template <typename T, int DH, bool WT, int WPR>
__global__ void __launch_bounds__(MG_THREADS) merge_kernel(Kv8Attn a, int RT, int grid) {
  using sm100::ex2;
  constexpr int PER = DH / 32;  // channels per lane
  constexpr int NW = MG_THREADS / 32;
  __shared__ long long sCount[NW][2];
  __shared__ float sStat[NW][3], sX[NW][DH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int R = a.G * a.n, nrg = (R + RT - 1) / RT, upb = a.c.Hkv * nrg;
  const int row = blockIdx.x * (NW / WPR) + warp / WPR, g = blockIdx.y, b = blockIdx.z, rg = row / RT, r = row % RT;
  const int u = g * nrg + rg;
  allow_next_kernel();
  const Tiles ts = unit_tiles(a, b);  // (lens is older than the attention, which waited before it started)
  long long before = 0, total = 0;
  for (int i = threadIdx.x; i < a.c.B; i += MG_THREADS) {
    const long long t = (long long)unit_tiles(a, i).n * upb;
    total += t;
    if (i < b) before += t;
  }
  before = warp_sum_ll(before);
  total = warp_sum_ll(total);
  if (lane == 0) {
    sCount[warp][0] = before;
    sCount[warp][1] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    before += sCount[i][0];
    total += sCount[i][1];
  }
  Records rec = {};
  if (ts.n && row < R) rec = unit_records(a, RT, DH, grid, before, total, b, u, upb, ts.n);
  // every CTA waits, so that this kernel's end means the attention's too
  wait_previous_kernel();
  if constexpr (WT) {
    const int rows = (R + NW / WPR - 1) / (NW / WPR);  // blocks of rows
    if (blockIdx.x >= rows) {
      if (WG_TILES * (blockIdx.x - rows) < ts.n) add_weights(a, RT, DH, grid, before, total, blockIdx.x - rows, g, b, ts);
      return;
    }
  }
  if (row >= R) return;  // (WPR 8: never; WPR 1: no barrier follows)
  T* out = (T*)a.out + ((size_t)b * a.n + row / a.G) * (size_t)(a.c.Hkv * a.G * DH) + (size_t)(g * a.G + row % a.G) * DH +
           lane * PER;
  if (ts.n == 0) {
#pragma unroll
    for (int k = 0; k < PER; ++k) out[k] = from_f<T>(0.f);
    return;
  }
  const int nrec = rec.n;
  if (nrec == 1) return;  // written whole by its CTA
  const size_t step = rec.step;
  const float* rec0 = rec.p + (size_t)r * (DH + 4);
  // this warp's records sub, sub + WPR, ..: 32 at a time, a lane's header each
  float L = -INFINITY, U = -INFINITY, sum = 0.f, x[PER] = {};
  for (int base = sub; base < nrec; base += 32 * WPR) {
    const int i = base + lane * WPR;
    const float4 h = i < nrec ? *(const float4*)(rec0 + i * step) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    const float nl = fmaxf(L, warp_max(h.x)), nu = fmaxf(U, warp_max(h.z));
    const float fl = L == -INFINITY ? 1.f : ex2(L - nl), fu = U == -INFINITY ? 1.f : ex2(U - nu);
    L = nl;
    U = nu;
    sum = sum * fl + warp_sum(h.x == -INFINITY ? h.y : h.y * ex2(h.x - L));
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] *= fu;
    const float f = h.z == -INFINITY ? 1.f : ex2(h.z - U);
    const int m = min(32, (nrec - base + WPR - 1) / WPR);
#pragma unroll 8
    for (int k = 0; k < m; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      const float* p = rec0 + (size_t)(base + k * WPR) * step + 4 + lane * PER;
      if constexpr (PER == 4) {
        const float4 y = *(const float4*)p;
        x[0] += y.x * fk; x[1] += y.y * fk; x[2] += y.z * fk; x[3] += y.w * fk;
      } else {
        const float2 y = *(const float2*)p;
        x[0] += y.x * fk; x[1] += y.y * fk;
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      sStat[warp][0] = L;
      sStat[warp][1] = sum;
      sStat[warp][2] = U;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) sX[warp][lane * PER + k] = x[k];
    __syncthreads();
    if (warp != 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      L = fmaxf(L, sStat[i][0]);
      U = fmaxf(U, sStat[i][2]);
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      sum += sStat[i][0] == -INFINITY ? sStat[i][1] : sStat[i][1] * ex2(sStat[i][0] - L);
      const float f = sStat[i][2] == -INFINITY ? 1.f : ex2(sStat[i][2] - U);
#pragma unroll
      for (int k = 0; k < PER; ++k) x[k] += sX[i][lane * PER + k] * f;
    }
  }
  const Norm f = row_norm(L, U, sum);
#pragma unroll
  for (int k = 0; k < PER; ++k) out[k] = from_f<T>(f(x[k]));
}

// ============================================================================ eviction
// Order of the weights as unsigned integers: larger float, larger key (NaN above infinity).
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 and 0 are equal
  return w != w ? 0xffffffffu : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// The kept positions.  A cluster of CTAs per (sequence, KV head); every lane owns KPT consecutive
// positions (a warp 32 KPT, a CTA 1024 KPT, rounds of them where the cluster's share is longer than that).
// Three passes of 11, 11 and 10 bits find the key of the last kept token among the middle ones
// [first, len - recent): each counts the digits of the keys that match the digits found so far, and a warp of
// every CTA adds the cluster's counts through distributed shared memory, first those of blocks of 64 digits,
// then those of the digits in the block that it needs (all 2048 of them, added in slices by the CTAs and
// handed back: 2.7 us more).  Then everyone counts what it keeps --
// forced tokens, keys above the found one, and of those equal to it the first `need` in position order --
// and after a prefix sum over lanes, warps and CTAs writes it in order.  Keys are loaded coalesced and
// turned to their owners through shared memory; a lane's matches are bits of one word, so that a token
// costs a few instructions a pass.  Bound by the chain of passes and cluster barriers: 8 heads of 131072
// positions about 12 us (one CTA per head, four passes of atomics: 390 us).
constexpr int SEL_THREADS = 1024, SEL_WARPS = SEL_THREADS / 32, SEL_BINS = 2048, SEL_CLUSTER = 8;
constexpr int KPT = 16;                     // positions per lane and round
constexpr int SEL_ROUND = SEL_THREADS * KPT;
constexpr int SEL_PITCH = 32 * (KPT + 1);   // a warp's keys in shared memory, one word of padding per lane
constexpr int SEL_SMEM = SEL_WARPS * SEL_PITCH * 4;

// Two neighbouring ints of this CTA's shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ int2 load_remote2(const int* p, uint32_t rank) {
  int2 v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\tld.shared::cluster.v2.b32 {%0, %1}, [r];\n\t}"
               : "=r"(v.x), "=r"(v.y) : "r"(sm100::smem_u32(p)), "r"(rank) : "memory");
  return v;
}
__device__ __forceinline__ int load_remote(const int* p, uint32_t rank) {
  int v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.b32 %0, [r];\n\t}"
               : "=r"(v) : "r"(sm100::smem_u32(p)), "r"(rank) : "memory");
  return v;
}
__device__ __forceinline__ int warp_excl(int v, int lane) {  // exclusive prefix sum over the lanes
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// Bits [lo, hi) of a word of KPT bits, bounds clamped.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), KPT);
  hi = min(max(hi, lo), KPT);
  return ((1u << hi) - 1u) & ~((1u << lo) - 1u);
}

__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const float* weights, int Lmax, int Hkv, int CL, const int* lens,
                                                             int keep, int first, int recent, int* kept, int* lens2) {
  extern __shared__ uint32_t skeys[];
  // this CTA's counts of digits and of blocks of 64 digits; a pass takes the one buffer while others may still
  // read the one of the pass before
  __shared__ __align__(8) int counts[2][SEL_BINS];
  __shared__ int blocks[2][SEL_WARPS];
  __shared__ __align__(8) int sTot[2];
  __shared__ int sWarp[2][SEL_WARPS], sPick[3];
  const int hd = blockIdx.x / CL, rank = blockIdx.x % CL, b = hd / Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  allow_next_kernel();
  wait_previous_kernel();
  const int len = min(max(lens[b], 0), Lmax);
  const float* w = weights + (size_t)hd * Lmax;
  int* out = kept + (size_t)hd * keep;
  if (threadIdx.x == 0 && rank == 0 && hd % Hkv == 0) lens2[b] = min(len, keep);
  if (len <= keep) {  // all of a short sequence (every CTA of the cluster takes this way)
    for (int i = rank * SEL_THREADS + threadIdx.x; i < keep; i += CL * SEL_THREADS) {
      out[i] = i < len ? i : -1;
    }
    return;
  }
  // this CTA's positions [cb, ce), in rounds of SEL_ROUND; a lane's of round q start at cb + q SEL_ROUND +
  // (32 warp + lane) KPT
  const int share = ((len + CL - 1) / CL + SEL_WARPS * KPT - 1) / (SEL_WARPS * KPT) * (SEL_WARPS * KPT);
  const int cb = min(rank * share, len), ce = min(cb + share, len), rounds = (ce - cb + SEL_ROUND - 1) / SEL_ROUND;
  const int m0 = first, m1 = len - recent;
  uint32_t* mine = skeys + warp * SEL_PITCH;
  const uint32_t* own = mine + lane * (KPT + 1);
  // a warp's keys of round q into shared memory (whole warp)
  auto load = [&](int q) {
    const int wb = cb + q * SEL_ROUND + warp * 32 * KPT;
    float f[KPT];
#pragma unroll
    for (int j = 0; j < KPT; ++j) f[j] = wb + j * 32 + lane < ce ? w[wb + j * 32 + lane] : 0.f;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int x = j * 32 + lane;
      mine[x + x / KPT] = weight_key(f[j]);
    }
    __syncwarp();
  };
  const bool once = rounds <= 1;  // the keys stay in shared memory from pass to pass
  for (int i = threadIdx.x; i < 2 * SEL_BINS; i += SEL_THREADS) counts[0][i] = 0;
  if (once) load(0);
  __syncthreads();
  int need = keep - first - recent;  // of the middle tokens; fewer than there are
  const bool none = need == 0;
  int low = 0;
  uint32_t prefix = 0, match = 0;  // match (once): this lane's middle positions that match the digits so far
  for (int pass = 0; pass < 3 && !none; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1;
    int *hist = counts[pass & 1], *block = blocks[pass & 1];
    for (int q = 0; q < rounds; ++q) {
      const int p = cb + q * SEL_ROUND + (warp * 32 + lane) * KPT;
      if (!once) load(q);
      if (!once || pass == 0) match = bit_range(m0 - p, min(m1, ce) - p);
      if (pass > 0) {
        uint32_t same = 0;
#pragma unroll
        for (int j = 0; j < KPT; ++j) same |= (own[j] >> (shift + bits)) == prefix ? 1u << j : 0u;
        match &= same;
      }
      if (pass == 0) {
#pragma unroll
        for (int j = 0; j < KPT; ++j)
          if ((match >> j) & 1) atomicAdd(&hist[own[j] >> 21], 1);
      } else {
        for (uint32_t m = match; m; m &= m - 1) atomicAdd(&hist[(own[__ffs(m) - 1] >> shift) & mask], 1);
      }
    }
    __syncthreads();
    {  // the blocks' counts, a warp each
      const int2 c = *(const int2*)(hist + 2 * threadIdx.x);
      const int n = __reduce_add_sync(0xffffffffu, c.x + c.y);
      if (lane == 0) block[warp] = n;
    }
    sm100::cluster_sync();
    if (warp == 0) {  // from the largest digit down: the block where the sum over the cluster reaches need, then its digit
      int n[SEL_CLUSTER], sum = 0;
#pragma unroll
      for (int r = 0; r < SEL_CLUSTER; ++r) n[r] = r < CL ? load_remote(block + 31 - lane, r) : 0;
#pragma unroll
      for (int r = 0; r < SEL_CLUSTER; ++r) sum += n[r];
      int before = warp_excl(sum, lane);
      const int at = (__ffs(__ballot_sync(0xffffffffu, before < need && need <= before + sum)) - 1) & 31;
      before = __shfl_sync(0xffffffffu, before, at);
      const int d = (31 - at) * 64 + 63 - 2 * lane;  // two digits a lane, d and d - 1
      int2 x[SEL_CLUSTER], c = make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < SEL_CLUSTER; ++r) x[r] = r < CL ? load_remote2(hist + d - 1, r) : make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < SEL_CLUSTER; ++r) {
        c.x += x[r].x;
        c.y += x[r].y;
      }
      before += warp_excl(c.x + c.y, lane);
      if (before < need && need <= before + c.x + c.y) {  // one lane
        const bool second = need > before + c.y;
        sPick[0] = second ? d - 1 : d;
        sPick[1] = need - before - (second ? c.y : 0);
        sPick[2] = second ? c.x : c.y;
      }
    } else if (pass == 1) {  // for the third pass; nobody reads this buffer behind the barrier above
      for (int i = threadIdx.x - 32; i < SEL_BINS; i += SEL_THREADS - 32) counts[0][i] = 0;
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)sPick[0];
    need = sPick[1];
    low = shift;
    if (need == sPick[2]) break;  // all of the bin is kept: the digits below do not matter
  }
  // prefix: the upper bits (above `low`) of the key of the last kept middle token, mostly 22 of them; need:
  // how many with exactly those.  A lane's sure
  // positions (forced, or above the key) and tied ones as bits, and their counts before it in its warp
  auto bits_of = [&](int p, uint32_t& sure, uint32_t& tie) {
    const uint32_t in = bit_range(0, ce - p), mid = bit_range(m0 - p, min(m1, ce) - p);
    uint32_t above = 0, equal = 0;
    if (!none) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const uint32_t k = own[j] >> low;
        above |= k > prefix ? 1u << j : 0u;
        equal |= k == prefix ? 1u << j : 0u;
      }
    }
    sure = in & (~mid | above);
    tie = mid & equal;
  };
  int nkeep = 0, ntie = 0;
  uint32_t su = 0, ti = 0;
  for (int q = 0; q < rounds; ++q) {
    if (!once) load(q);
    bits_of(cb + q * SEL_ROUND + (warp * 32 + lane) * KPT, su, ti);
    nkeep += __popc(su);
    ntie += __popc(ti);
  }
  // (over all rounds of a CTA; with several rounds the warps' parts interleave and are ordered below)
  nkeep = __reduce_add_sync(0xffffffffu, nkeep);
  ntie = __reduce_add_sync(0xffffffffu, ntie);
  if (lane == 0) {
    sWarp[0][warp] = nkeep;
    sWarp[1][warp] = ntie;
  }
  __syncthreads();
  if (warp == 0) {
    nkeep = __reduce_add_sync(0xffffffffu, sWarp[0][lane]);
    ntie = __reduce_add_sync(0xffffffffu, sWarp[1][lane]);
    if (lane == 0) {
      sTot[0] = nkeep;
      sTot[1] = ntie;
    }
  }
  sm100::cluster_sync();
  int kb = 0, tb = 0;  // sure ones and ties before the current round
  int2 tot[SEL_CLUSTER];
#pragma unroll
  for (int r = 0; r < SEL_CLUSTER; ++r) tot[r] = r < rank ? load_remote2(sTot, r) : make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < SEL_CLUSTER; ++r) {
    kb += tot[r].x;
    tb += tot[r].y;
  }
  sm100::cluster_arrive();  // no CTA leaves while another reads its counts
  for (int q = 0; q < rounds; ++q) {
    const int p = cb + q * SEL_ROUND + (warp * 32 + lane) * KPT;
    if (!once) {
      load(q);
      bits_of(p, su, ti);
    }
    int k = warp_excl(__popc(su), lane), t = warp_excl(__popc(ti), lane);
    __syncthreads();
    if (lane == 31) {
      sWarp[0][warp] = k + __popc(su);
      sWarp[1][warp] = t + __popc(ti);
    }
    __syncthreads();
    const int a0 = sWarp[0][lane], a1 = sWarp[1][lane];
    k += kb + __shfl_sync(0xffffffffu, warp_excl(a0, lane), warp);
    t += tb + __shfl_sync(0xffffffffu, warp_excl(a1, lane), warp);
    kb += __reduce_add_sync(0xffffffffu, a0);
    tb += __reduce_add_sync(0xffffffffu, a1);
    for (uint32_t m = su | ti; m; m &= m - 1) {
      const int j = __ffs(m) - 1, i = p + j;
      const bool tied = (ti >> j) & 1;
      const int at = k + min(t, need);
      if ((!tied || t < need) && at < keep) out[at] = i;
      k += !tied;
      t += tied;
    }
  }
  sm100::cluster_wait();
}

// Kept rows into the new cache, a token block at a time: one CTA per (block, K or V and head, sequence).
// The largest magnitude is found on the codes themselves (their low 7 bits order like the values), a
// chunk at a time with its own scale, and codes whose scale stays are copied as they are.  Rows come one by
// one (128 bytes): 8 heads, 8192 rows: 34 MB in about 9 us, bound by the chain kept - code.
template <int DH, int CH>
__global__ void __launch_bounds__(AP_THREADS) compact_kernel(Kv8Args a, Kv8Args d, const int* kept, int keep,
                                                      const float* weights, float* weights2) {
  __shared__ float red[AP_THREADS / 32];
  constexpr int CPR = DH / 16;
  const int b = blockIdx.z, kv = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
  allow_next_kernel();
  wait_previous_kernel();
  // (`kept` is -1 behind a short sequence's positions: dst_lens need not be read first)
  const int t0 = blockIdx.x * d.block, rows = min(d.block, keep - t0);
  const size_t hd = (size_t)b * a.Hkv + g;
  const uint8_t* src = (const uint8_t*)(kv ? a.v : a.k) + hd * a.Lmax * DH;
  const float* ss = (kv ? a.vs : a.ks) + hd * a.nblk;
  uint8_t* dst = (uint8_t*)(kv ? d.v : d.k) + (hd * d.Lmax + t0) * DH;
  if (!kv && weights2 && threadIdx.x < rows) {
    const int from = kept[hd * keep + t0 + threadIdx.x];
    if (from >= 0) weights2[hd * d.Lmax + t0 + threadIdx.x] = weights[hd * a.Lmax + from];
  }
  int j[CH];
  uint4 v[CH];
  float sc[CH], m = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int ch = i * AP_THREADS + threadIdx.x;
    j[i] = ch < rows * CPR ? kept[hd * keep + t0 + ch / CPR] : -1;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (j[i] >= 0) {
      v[i] = *(const uint4*)(src + (size_t)j[i] * DH + (i * AP_THREADS + threadIdx.x) % CPR * 16);
      sc[i] = ss[j[i] >> a.lb];
    }
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (j[i] >= 0) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t x = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t y = w[k] & 0x7f7f7f7fu;
        x = __vmaxu4(x, y & ~__vcmpeq4(y, 0x7f7f7f7fu));  // (NaN does not count)
      }
      x = __vmaxu4(x, x >> 16);
      m = fmaxf(m, e4m3x2_to_f2(max(x & 0xff, (x >> 8) & 0xff)).x * sc[i]);
    }
  m = block_max<AP_THREADS>(m, red);
  const int e = scale_exp(m);
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (j[i] >= 0) {
      if (exp_of(sc[i]) != e) v[i] = rescale16(v[i], exp_of(sc[i]) - e);
      *(uint4*)(dst + (size_t)(i * AP_THREADS + threadIdx.x) * 16) = v[i];
    }
  if (threadIdx.x == 0 && j[0] >= 0) (kv ? d.vs : d.ks)[hd * d.nblk + blockIdx.x] = pow2(e);
}

// Calls f(integral_constant) with the 16-value chunks per thread of a token block.
template <typename F>
cudaError_t with_chunks(int block, int dh, F f) {
  const int ch = (block * dh / 16 + AP_THREADS - 1) / AP_THREADS;
  if (ch <= 1) return f(std::integral_constant<int, 1>());
  if (ch <= 2) return f(std::integral_constant<int, 2>());
  if (ch <= 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 8>());
}

}  // namespace kv8

cudaError_t kv8_append(const Kv8Args& a, const void* kn, const void* vn, int is_bf16, long long row_stride,
                       long long batch_stride, int n, const int* pos, const int* count, int* status, cudaStream_t s) {
  const dim3 grid((n + a.block - 1 + a.block - 1) / a.block, 2 * a.Hkv, a.B);
  auto run = [&](auto dh) {
    constexpr int DH = decltype(dh)::value;
    return kv8::with_chunks(a.block, DH, [&](auto ch) {
      constexpr int CH = decltype(ch)::value;
      if (is_bf16)
        return launch_dependent(kv8::append_kernel<bf16, DH, CH>, grid, kv8::AP_THREADS, 0, s, a, (const bf16*)kn,
                                (const bf16*)vn, row_stride, batch_stride, n, pos, count, status);
      return launch_dependent(kv8::append_kernel<float, DH, CH>, grid, kv8::AP_THREADS, 0, s, a, (const float*)kn,
                              (const float*)vn, row_stride, batch_stride, n, pos, count, status);
    });
  };
  return a.dh == 128 ? run(std::integral_constant<int, 128>()) : run(std::integral_constant<int, 64>());
}

cudaError_t kv8_read(const Kv8Args& a, const int* first, const int* rows, int n, void* k_out, void* v_out, int is_bf16,
                     long long row_stride, long long batch_stride, int* status, cudaStream_t s) {
  const int chunks = n * (a.dh / 16);  // of one head
  auto run = [&](auto type, auto dh, auto nc) {
    using T = decltype(type);
    constexpr int NC = decltype(nc)::value;
    const dim3 grid((chunks + 256 * NC - 1) / (256 * NC), 2 * a.Hkv, a.B);
    return launch_dependent(kv8::read_kernel<T, decltype(dh)::value, NC>, grid, 256, 0, s, a, first, rows, n, (T*)k_out,
                            (T*)v_out, row_stride, batch_stride, status);
  };
  // two chunks a thread once that still leaves every SM four blocks; fewer rows: more threads
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  auto with_nc = [&](auto type, auto dh) {
    return (long long)chunks * 2 * a.Hkv * a.B >= 2 * 256 * 4LL * sms ? run(type, dh, std::integral_constant<int, 2>())
                                                                    : run(type, dh, std::integral_constant<int, 1>());
  };
  auto with_dh = [&](auto type) {
    return a.dh == 128 ? with_nc(type, std::integral_constant<int, 128>()) : with_nc(type, std::integral_constant<int, 64>());
  };
  return is_bf16 ? with_dh(bf16()) : with_dh(float());
}

// Groups of 8 query rows per unit: a second one shares the cache's bytes and conversions.
static int kv8_groups(int R) { return R <= 8 ? 1 : 2; }
// CTAs: as many as the registers and the stages (d_head 128: 65 KB a CTA) let stay resident.
static int kv8_grid(int R, int dh) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int grid = sms * (kv8_groups(R) == 2 && dh == 128 ? 2 : 3);
  return grid < kv8::MG_MOST ? grid : kv8::MG_MOST;
}

size_t kv8_attention_scratch(const Kv8Args& c, int G, int n, int weights, size_t* stats, size_t* scores) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t R = (size_t)G * n, RT = 8 * kv8_groups((int)R), nrg = (R + RT - 1) / RT;
  size_t o = al((kv8_grid((int)R, c.dh) + (size_t)c.B * c.Hkv * nrg) * RT * (c.dh + 4) * 4);
  *stats = o;
  if (weights) o += al((size_t)c.B * c.Hkv * R * 8);
  *scores = o;
  if (weights) o += al((size_t)c.B * c.Hkv * c.Lmax * nrg * RT * 4);
  return o;
}

cudaError_t kv8_attention(const Kv8Attn& a, int is_bf16, int* status, cudaStream_t s) {
  const int R = a.G * a.n, nt = kv8_groups(R), most = kv8_grid(R, a.c.dh);
  const long long units = (long long)a.c.B * a.c.Hkv * ((R + 8 * nt - 1) / (8 * nt));
  // Few ranges per unit: a warp joins a row.  Otherwise a CTA does, and the attention leaves a few CTAs'
  // room free, so that those CTAs are in place and past their prologue when it ends (1 x 131072, 28/4
  // heads: 36.0 -> 32.5 us)
  const bool few = most <= 8 * units;
  const int grid = few ? most : most - (int)(R * units / 2 + 1 < most / 16 ? R * units / 2 + 1 : most / 16);
  const long long rows = (long long)a.c.B * a.c.Hkv * a.c.Lmax;
  CUtensorMap tk, tv;
  cudaError_t me = make_tmap_u8(&tk, a.c.k, rows, a.c.dh, 32);
  if (me == cudaSuccess) me = make_tmap_u8(&tv, a.c.v, rows, a.c.dh, 32);
  if (me != cudaSuccess) return me;
  auto run = [&](auto type, auto dh, auto nts, auto wt) {
    using T = decltype(type);
    constexpr int DH = decltype(dh)::value, NT = decltype(nts)::value;
    constexpr bool WT = decltype(wt)::value;
    auto* kernel = kv8::attention_kernel<T, DH, NT, WT>;
    constexpr int smem = kv8::AtCfg<DH>::SMEM;
    cudaError_t e = raise_max_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(kernel, grid, kv8::AT_THREADS, smem, s, tk, tv, a, status)) != cudaSuccess) return e;
    const int rows = few ? (R + 7) / 8 : R, tokens = WT ? (a.c.Lmax + kv8::WG_TILES * kv8::TILE - 1) / (kv8::WG_TILES * kv8::TILE) : 0;
    return launch_dependent(few ? kv8::merge_kernel<T, DH, WT, 1> : kv8::merge_kernel<T, DH, WT, 8>,
                            dim3(rows + tokens, a.c.Hkv, a.c.B), kv8::MG_THREADS, 0, s, a, 8 * NT, grid);
  };
  auto with_wt = [&](auto type, auto dh, auto nts) {
    return a.weights ? run(type, dh, nts, std::true_type()) : run(type, dh, nts, std::false_type());
  };
  auto with_nt = [&](auto type, auto dh) {
    return nt == 1 ? with_wt(type, dh, std::integral_constant<int, 1>())
                   : with_wt(type, dh, std::integral_constant<int, 2>());
  };
  auto with_dh = [&](auto type) {
    return a.c.dh == 128 ? with_nt(type, std::integral_constant<int, 128>())
                         : with_nt(type, std::integral_constant<int, 64>());
  };
  return is_bf16 ? with_dh(bf16()) : with_dh(float());
}

cudaError_t kv8_evict(const Kv8Args& a, const int* lens, const float* weights, int keep, int first, int recent,
                      const Kv8Args& d, int* lens2, float* weights2, int* kept, cudaStream_t s) {
  // CTAs per head: as few as take a head in one round each, at most 8 (portable).  A CTA (1024 threads of 64
  // registers) fills an SM, 148, 74, 33 and 15 clusters of 1, 2, 4 and 8 fit the card, and a second round costs
  // more than idle SMs or a second wave do.  The call with 1 / 2 / 4 / 8 CTAs a head, in us: 16 heads of 16384
  // positions 13.9 / 14.2 / 14.4 / -, of 65536 49.2 / 30.2 / 14.4 / 25.1; 64 heads of 32768 32.8 / 17.7 / 29.2 /
  // 60.2; 32 heads of 131072 106 / 60 / 40 / 37; the other way round only at 256 heads of 131072, 198 / 199 / 231 / 209.
  int cl = 1;
  while (cl < kv8::SEL_CLUSTER && cl * kv8::SEL_ROUND < a.Lmax) cl *= 2;
  cudaError_t e = raise_max_smem(kv8::select_kernel, kv8::SEL_SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(a.B * a.Hkv * cl);
  lc.blockDim = dim3(kv8::SEL_THREADS);
  lc.dynamicSmemBytes = kv8::SEL_SMEM;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  e = cudaLaunchKernelEx(&lc, kv8::select_kernel, weights, a.Lmax, a.Hkv, cl, lens, keep, first, recent, kept, lens2);
  if (e != cudaSuccess) return e;
  const dim3 grid((keep + d.block - 1) / d.block, 2 * a.Hkv, a.B);
  auto run = [&](auto dh) {
    constexpr int DH = decltype(dh)::value;
    return kv8::with_chunks(d.block, DH, [&](auto ch) {
      return launch_dependent(kv8::compact_kernel<DH, decltype(ch)::value>, grid, kv8::AP_THREADS, 0, s, a, d, (const int*)kept, keep,
                              weights, weights2);
    });
  };
  return a.dh == 128 ? run(std::integral_constant<int, 128>()) : run(std::integral_constant<int, 64>());
}

}  // namespace mka
