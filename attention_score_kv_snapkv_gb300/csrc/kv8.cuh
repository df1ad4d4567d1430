// The 8-bit KV cache (KVC_KV8_BLOCK rows of one unit share one power-of-two scale): launch
// arguments of its kernels and the quantisation both the writers and the decode step use.
#pragma once

#include <cuda_fp16.h>

#include "kvc_internal.cuh"

namespace kvc {

constexpr int KB8 = KVC_KV8_BLOCK;  // rows of one scale
constexpr int KL8 = KB8 + 1;        // rows of a unit in k_last and v_last

// The cache as the kernels see it.
struct Kv8 {
  uint8_t *kq, *vq;            // [U, cap, D] e4m3 codes
  float *ks, *vs;              // [U, cap / KB8] scales (powers of two)
  __nv_bfloat16 *kt, *vt;      // [U, KB8, D] the rows past the last whole block
  int32_t *pos;                // [U, cap] or null
  int32_t *n_valid;            // [U]
  // What lets a row count be lowered into a block that has been quantised since (all null: it may
  // not be): the rows of the block that was completed last, as they came, and behind them a copy
  // of the tail's first row as the last call left it; and for each unit x the block that the
  // tail's rows belong to, y the block held here (-1: none).
  __nv_bfloat16 *kl, *vl;      // [U, KL8, D]
  int2 *blocks;                // [U]
  int units, D, cap;
};

// Where the rows of the block that n rows leave open are: in the tail, in kl and vl, or nowhere
// any more.  The latter two only if the tail's first row is still the one that the last call
// left: a tail that the caller has put other rows into is taken as it is.
enum : int { OPEN_TAIL = 0, OPEN_LAST = 1, OPEN_GONE = 2 };
__device__ __forceinline__ int open_rows(int n, int2 blk) {
  if (n % KB8 == 0 || blk.x <= n / KB8) return OPEN_TAIL;
  return blk.y == n / KB8 ? OPEN_LAST : OPEN_GONE;
}
__device__ __forceinline__ bool same16(uint4 a, uint4 b) {
  return ((a.x ^ b.x) | (a.y ^ b.y) | (a.z ^ b.z) | (a.w ^ b.w)) == 0;
}

struct Kv8WriteArgs {
  Kv8 c;
  const void *k, *v;           // [U, L, D] bf16
  const int32_t *rows;         // [U, rows_ld] source row of each cache row, or null: row r
  int rows_ld;
  const int32_t *pos_in;       // [U, n_rows] positions to record, or null: the source row
  const int32_t *lengths;      // [U] rows written of each unit, or null: n_rows
  int L, n_rows;
  int set_state;               // 1: also write pos and n_valid
};
struct Kv8AppendArgs {
  Kv8 c;
  const void *k, *v;           // [U, m, D] bf16
  const int32_t *counts;       // [U] or null: m
  int m, new_pos;
  int *cnt;                    // [U] zero between calls
};
struct Kv8ReadArgs {
  Kv8 c;
  void *k, *v;                 // [U, out_rows, D] bf16
  int out_rows;
};
struct Kv8DecodeArgs {
  Kv8 c;
  const void *q;               // [U * G, D]
  const void *k_new, *v_new;   // [U, D] or null
  void *out;                   // [U * G, D]
  void *ws;
  int G, new_pos;
};
cudaError_t launch_kv8_write(const Ctx &c, const Kv8WriteArgs &a);
cudaError_t launch_kv8_append(const Ctx &c, const Kv8AppendArgs &a);
cudaError_t launch_kv8_read(const Ctx &c, const Kv8ReadArgs &a);
cudaError_t launch_kv8_decode(const Ctx &c, const Kv8DecodeArgs &a);
size_t kv8_decode_ws_bytes(long long units, int G, int D);
int *kv8_unit_counts(void *ws);  // [U] counts at zero between calls

// kvc_api.cu: the current device's launch context (and the tensor-map encoder loaded).
kvc_status make_ctx(kvc_stream_t stream, Ctx *c);
// kvc_api.cu: a tensor map over rows of 128 bytes, boxes of box_rows whole rows, with the
// 128-byte swizzle.
bool encode_bytes_map(CUtensorMap *map, const void *base, uint64_t rows, int box_rows);
// kvc_api.cu: SnapKV's votes (or the given ones) and selection, positions and row counts
// only; *v_dev receives v's device address (v may be page-locked host memory).
kvc_status snapkv_positions(const kvc_snapkv_params *p, const void *q_win, const float *votes,
                            const void *k, const void *v, int32_t *pos_out, int32_t *n_valid_out,
                            float *votes_out, void *workspace, size_t workspace_bytes,
                            kvc_stream_t stream, const void **v_dev);

// A bounded wait whose first test is all that a barrier that is ready costs; the rest is kept
// out of line, and what only it needs in shared memory, for the warps' code competes for the
// instruction cache.
struct WaitState {
  int flag;  // raised by the first wait of the CTA that runs out
  uint32_t *status;
  unsigned long long limit;
};
inline __device__ __noinline__ bool wait_all_slow(WaitState *s, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, Abort{&s->flag, s->status, s->limit}.wait(bar, parity));
}
struct Wait {
  WaitState *s;  // in shared memory
  // by a whole warp, which agrees
  __device__ __forceinline__ bool all(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_all_slow(s, bar, parity);
  }
};
// For the copies and products in flight at the end, whatever became of the rest: a millisecond at
// least, however short the limit.
inline __device__ __noinline__ void wait_drain(uint32_t bar, uint32_t parity, unsigned long long limit) {
  mbar_wait_bounded(bar, parity, limit < 1000000ull ? 1000000ull : limit);
}

// Barrier of `nthreads` threads that also tells whether `v` holds in all of them.
__device__ __forceinline__ bool all_of(int id, int nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------------------
// Quantisation of one block.  amax: the bit pattern (bf16, sign cleared) of the block's
// largest finite magnitude.  The scale is the least power of two 2^e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8 is e4m3's largest value), so x / scale and code * scale are exact and
// the only rounding is the one to 4 significant bits (half a step: 2^-4 relative; values
// under 2^-6 of the scale: 2^-10 of it).  -126 <= e keeps 2^-e finite; bf16 magnitudes that
// small are multiples of 2^-133, which codes at 2^-126 still hold to 2^-135.
// ------------------------------------------------------------------------------
__device__ __forceinline__ int kv8_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7f) > 0x60 ? 1 : 0);
  return max(e, -126);  // amax <= 0x7f7f gives e <= 120
}
__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two floats to two e4m3 codes (lo in the low byte), round to nearest even; NaN -> 0x7f.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes to two floats (exact).
__device__ __forceinline__ float2 e4m3x2_float(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The largest magnitude of the packed bf16 pairs seen so far, both halves apart; bit
// patterns order as the values do, and infinities and NaN (>= 0x7f80) order above them.
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, uint4 w) {
  m = __vmaxu2(m, w.x & 0x7fff7fffu);
  m = __vmaxu2(m, w.y & 0x7fff7fffu);
  m = __vmaxu2(m, w.z & 0x7fff7fffu);
  return __vmaxu2(m, w.w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {  // non-finite halves -> 0
  w &= 0x7fff7fffu;
  if ((w & 0xffffu) >= 0x7f80u) w &= 0xffff0000u;
  if ((w >> 16) >= 0x7f80u) w &= 0xffffu;
  return w;
}

// Eight bf16 values to eight codes.
__device__ __forceinline__ uint2 encode8(uint4 w, float inv) {
  uint2 r;
  r.x = e4m3x2(bf_lo(w.x) * inv, bf_hi(w.x) * inv) | (e4m3x2(bf_lo(w.y) * inv, bf_hi(w.y) * inv) << 16);
  r.y = e4m3x2(bf_lo(w.z) * inv, bf_hi(w.z) * inv) | (e4m3x2(bf_lo(w.w) * inv, bf_hi(w.w) * inv) << 16);
  return r;
}
// The same where the block holds a non-finite value (coded as NaN: e4m3 has no infinity)
// or values so large (e = 120) that a code above `lim` would read back as infinity.
__device__ __forceinline__ uint32_t encode1_rare(uint32_t half, float inv, float lim) {
  const uint32_t mag = half & 0x7fffu;
  if (mag >= 0x7f80u) return 0x7fu;
  const float x = __uint_as_float(half << 16) * inv;
  return e4m3x2(fminf(fmaxf(x, -lim), lim), 0.f) & 0xffu;
}
inline __device__ __noinline__ uint2 encode8_rare(uint4 w, float inv, float lim) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    out[i >> 2] |= encode1_rare((in[i >> 1] >> ((i & 1) * 16)) & 0xffffu, inv, lim) << ((i & 3) * 8);
  return make_uint2(out[0], out[1]);
}

constexpr int KV8_NT = 128;  // threads that quantise one block of K or V

// Quantises one block whose rows the 128 threads hold (thread t: pieces t, t + 128, ... of
// eight values, piece = row * D / 8 + column / 8): codes to dst [KB8, D], the scale to
// *scale.  red: 4 words of shared memory, bar: a named barrier of these 128 threads.
template <int D>
__device__ __forceinline__ void quantise_block(const uint4 (&w)[KB8 * D / 8 / KV8_NT], uint8_t *dst,
                                               float *scale, uint32_t *red, int bar, int t) {
  constexpr int NP = KB8 * D / 8 / KV8_NT;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) m = amax_bits(m, w[i]);
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if ((t & 31) == 0) red[t >> 5] = m;
  named_bar(bar, KV8_NT);
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  named_bar(bar, KV8_NT);  // red may be rewritten
  const bool nonfinite = m >= 0x7f80u;
  if (nonfinite) {  // the scale comes from the finite values alone
    m = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      m = amax_bits(m, make_uint4(finite_bits(w[i].x), finite_bits(w[i].y), finite_bits(w[i].z),
                                  finite_bits(w[i].w)));
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if ((t & 31) == 0) red[t >> 5] = m;
    named_bar(bar, KV8_NT);
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    named_bar(bar, KV8_NT);
  }
  const int e = kv8_exponent(m);
  const float inv = exp2_int(-e);
  uint2 *out = reinterpret_cast<uint2 *>(dst);
  if (nonfinite || e == 120) {
    const float lim = e == 120 ? 240.f : 448.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) out[t + i * KV8_NT] = encode8_rare(w[i], inv, lim);
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) out[t + i * KV8_NT] = encode8(w[i], inv);
  }
  if (t == 0) *scale = exp2_int(e);
}

}  // namespace kvc
