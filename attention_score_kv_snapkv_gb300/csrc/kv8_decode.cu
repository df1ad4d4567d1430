// Decode attention over the 8-bit KV cache: for each query head of each (layer, batch, KV
// head) unit, o = softmax(q . K^T / sqrt(D)) . V over the unit's n rows, the whole blocks in
// e4m3 codes with a scale a block, the last n mod 64 rows in bf16; with an optional append.
//
// HBM-bound (2 D bytes a row against 4 G D flop), so the codes are never widened: both
// products run on the tensor cores straight from the e4m3 tiles that TMA brings in.
//
// * S^T = K . q^T (tcgen05 kind::f8f6f4, 128 keys x 16 columns): q is split, exactly but for
//   elements under 2^-14 of the head's largest (2^-21 of it at most is lost), into two e4m3
//   terms, q 2^-e = hi + lo / 16 (bf16 has 8 significant bits, e4m3 holds 4, and the rounded
//   remainder fits 4), which take a column each; the logit is (hi + lo / 16) 2^e scale_k.
// * O^T = V^T . P^T (128 lanes x 16 or 32 columns): a weight is rounded to fp16 (11 bits: off by at
//   most 2^-11 of itself) and split the same way into three e4m3 terms, a column each.  The weight
//   of key j in a tile is exp2(s_j + log2 scale_v - M) with M the tile's largest s_j + log2 scale_v,
//   so V's scale costs nothing and blocks of very different sizes lose no bits to each other.  (A
//   block of zeros has the scale 1, which says nothing of its size: it is looked for, and counts
//   with the least.)  A tile's product is not accumulated in tensor memory: four warps read it, one
//   lane a thread, and add it to their registers with the running maximum's factor, so nothing in
//   tensor memory is ever rescaled, and a weight keeps its 11 bits down to 2^-14 of its own tile's
//   largest and is off by at most 2^-26 of it below that.
// * D = 64 lies two keys to a 128-byte row: a tile is then 256 keys, S takes two products (the
//   rows' first and second halves), and one O product serves both, lanes 0-63 the first keys,
//   64-127 the second, each half of the lanes reading its half of the columns.
// * The tail's tile goes through the same pipeline with bf16 operands (kind::f16): q as it is,
//   the weights in two bf16 terms.
// * The plan is made on the device, from the row counts, so ragged batches balance and the
//   capacity costs nothing.  The units' blocks, and a tile's worth of slots for each tail, form
//   one sequence that is split evenly over one CTA an SM; where the units are few, every CTA
//   instead takes up to C slots of one unit (U = 8, 300 rows: 8.0 us became 6.8).  A CTA takes its
//   last unit first, so that shared units are done early.  The last CTA to finish a shared unit
//   merges its segments: a warp of its own does while the others stream on (a fence and a count
//   take up to 5 us behind the tiles; in the queries' warp they cost 3 us of 34 at U = 512), or
//   the whole CTA at its end.
// * With an append every CTA reads the row counts before any changes: the last CTA to have
//   planned (an atomic count) advances them, while the others already stream.  The CTA that
//   has a unit's tail writes the new row, or quantises the block that it completes and keeps that
//   block's rows as they came; a row count lowered into that block has the tail's tile from there.
// * Every wait is bounded; one that runs out sets the device's timeout flag and the CTA drains.
//
// Warps: TMA; S; PV; queries; 2 x 4 softmax (alternate tiles); 4 output; merge.  Four tiles may
// lie between any two of them.
// Measured (GB300, graph of calls with the append on three caches in turn, against 6.68 TB/s of
// measured copy): 64 units of 131050 rows, G = 1: 310 us (2.15 GB, 104%); 512 units of 1100 rows,
// G = 4: 31.3 us (0.15 GB, 70%: 7 us are launch, plan, first tile and end, the rest runs at 6.6
// TB/s); 192 ragged units up to 8191 rows, D = 64, G = 8: 27.5 us (0.10 GB, 56%: short units' ends
// and the softmax's latency); 8 units of 300 rows: 7.2 us (latency).
#include <math.h>

#include "kv8.cuh"

namespace kvc {
namespace {

constexpr int TROWS = 128;      // 128-byte rows of a tile: one key each (D = 128) or two (D = 64)
constexpr int NWARP = 17;
constexpr int NTH = 32 * NWARP;
constexpr int W_TMA = 0, W_S = 1, W_PV = 2, W_Q = 3, W_SM = 4, W_OUT = 12, W_M = 16;
constexpr int MAXCTA = 192;     // CTAs the scratch has room for
constexpr int SNAP = 512;       // row counts a CTA keeps in shared memory
constexpr int MINC = 8;         // slots of a CTA that has one unit's share (the aligned plan), at least
constexpr int MINS = 2;         // slots a CTA takes at least in the streamed plan
constexpr int NB = 4;           // tiles between the two products and between P and the output
constexpr int TMEM_COLS = 512;
constexpr int T_S = 0, T_O = 32 * NB;  // tensor-memory columns: S [NB][32], O [NB][64]
constexpr int FEW = 4;          // segments that one thread merges by itself
constexpr int QN = 16;          // columns of the S product
constexpr int SB = TROWS * 128; // bytes of a stage: 128 rows in 8 bits, or 64 rows in bf16

template <int D, int G>
struct Geo {
  static constexpr int KPR = 128 / D;           // keys of a 128-byte row
  static constexpr int TB = 2 * KPR;            // blocks of a tile
  static constexpr int BR = KB8 / KPR;          // 128-byte rows of a block
  static constexpr int HB = G <= 4 ? 4 : 8;     // columns of one term
  static constexpr int PN = G <= 4 ? 16 : 32;   // columns of one key's terms (three of them)
  static constexpr int NST = D == 64 && G == 8 ? 10 : 12;  // stages; K in even ones, V in odd ones
  static constexpr int KBT = D / 64;            // 128-byte column blocks of a bf16 tail tile
  static constexpr int OFF_Q8 = NST * SB;                  // [2][16 rows][D]
  static constexpr int OFF_QT = OFF_Q8 + 2 * QN * D;       // [2][KBT][16 rows][128 B]
  static constexpr int OFF_P = OFF_QT + 2 * QN * D * 2;    // [NB] weights, 16 bytes a row and column group
  static constexpr int PB = TROWS * PN * KPR;
  static constexpr int OFF_X = OFF_P + NB * PB;             // float [64][G]: D = 64's second half
  static constexpr int OFF_SN = OFF_X + (D == 64 ? 64 * G * 4 : 0);  // int [SNAP]
  static constexpr int OFF_QS = OFF_SN + SNAP * 4;         // float [8][8] logit factors
  static constexpr int OFF_MX = OFF_QS + 8 * 8 * 4;        // float [2 sets][2][8][4] warp maxima
  static constexpr int OFF_MT = OFF_MX + 2 * 2 * 8 * 4 * 4;  // float [NB][8] tile references
  static constexpr int OFF_ST = OFF_MT + NB * 8 * 4;        // float2 [2][8 warps][8] (max, normaliser)
  static constexpr int OFF_BAR = OFF_ST + 2 * 8 * 8 * 8 + 8 * 16;  // and float4 [8]
  static constexpr int SMEM = OFF_BAR + 768 + 1024;
  static_assert(OFF_Q8 % 1024 == 0 && OFF_QT % 1024 == 0 && OFF_P % 1024 == 0, "operand alignment");
  static_assert(NST % 2 == 0 && SMEM <= 232448, "shared memory");
};

// barriers (bytes from OFF_BAR)
constexpr int B_FULL = 0;      // [NST <= 12] stage loaded
constexpr int B_EMPTY = 96;    // [NST] its MMAs are done
constexpr int B_SFULL = 192;   // [NB] S^T written
constexpr int B_SEMPTY = 224;  // [NB] and read
constexpr int B_PFULL = 256;   // [NB] weights written
constexpr int B_OFULL = 288;   // [NB] O^T written
constexpr int B_OEMPTY = 320;  // [NB] and read
constexpr int B_QFULL = 352;   // [2] a unit's queries
constexpr int B_QEMPTY = 368;  // [2]
constexpr int B_RFULL = 384;   // [2] a segment's normalisers are there
constexpr int B_REMPTY = 400;  // [2]
constexpr int B_START = 416;   // the first unit's small operands have arrived
constexpr int B_MISC = 424;    // ints
constexpr int M_WAIT = 0;      // the waits' state
constexpr int M_TMEM = 6, M_UF = 7, M_PF = 8, M_UL = 9, M_PL = 10, M_LAST = 11;
constexpr int M_WS = 12;       // [2][NWARP] plan: warp sums
constexpr int M_RED = 46;      // [4] quantisation
constexpr int M_VALID = 50;    // [2] a shared unit's segment was completed
constexpr int M_TODO = 52;     // [2][4] this CTA merges it at the end: the Shared (nseg 0: it does not)
static_assert(sizeof(WaitState) == 4 * (M_TMEM - M_WAIT) && B_MISC % 8 == 0, "the waits' state");
constexpr int M_RE = 60;       // [1 + SNAP / 32] whether, and which, units have their open rows in kl and vl
static_assert(B_MISC + 4 * (M_RE + 1 + SNAP / 32) <= 768, "barrier area");

struct P8 {
  const __nv_bfloat16 *q, *k_new, *v_new;
  __nv_bfloat16 *out;
  Kv8 c;
  float lc;                // log2(e) / sqrt(D)
  int ga, new_pos;
  int *planned;            // CTAs that have read the row counts
  int *cnt;                // [U] finished segments of a shared unit
  int *snap;               // [U] row counts before the append, negative (~n) with open rows in kl and vl
  float2 *part_ml;         // [2 * MAXCTA][G]
  float *part_o;           // [2 * MAXCTA][G][D]
  uint32_t *status;
  unsigned long long timeout;
};

__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
constexpr uint32_t L_NONE = 0, L_128B = 2, L_64B = 4;

// Instruction descriptors (D fp32, M = 128): e4m3 x e4m3 or bf16 x bf16; transposed operands
// are the ones that lie with their long side contiguous (MN-major).
__host__ __device__ constexpr uint32_t idesc8(int N, bool tr) {
  return (1u << 4) | (tr ? (1u << 15) | (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__host__ __device__ constexpr uint32_t idesc16(int N, bool tr) {
  return idesc_bf16(TROWS, N) | (tr ? (1u << 15) | (1u << 16) : 0u);
}

// The producer and the two MMA warps run converged, one elected lane issuing by predicate:
// their addresses and descriptors then stay in uniform registers.  (A branch on the lane cost
// 300 to 400 clocks a tile in each of them.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// x, of which the compiler knows nothing, so that it does not compile what follows once for each
// value: the warps' code together is more than an SM's instruction cache holds (without this, the
// loops that are kept rolled and the plan's results in shuffles, 1216 units of 544 rows, D = 64,
// 8 heads took 41 us, with it 30; 33 since rows can be taken back and zeros are looked for).
__device__ __forceinline__ bool opaque(bool x) {
  uint32_t r = x;
  asm volatile("" : "+r"(r));
  return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void mma_f8(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\t"
      "setp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t lead, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred l;\n\t"
      "setp.ne.b32 l, %2, 0;\n\t"
      "@l mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t lead, uint32_t dst, const CUtensorMap *map, int32_t x,
                                         int32_t y, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\t"
      "setp.ne.b32 l, %5, 0;\n\t"
      "@l cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y),
      "r"(bar), "r"(lead)
      : "memory");
}

__device__ __forceinline__ int slot_first(int b, int Q, int R) { return b * Q + min(b, R); }
__device__ __forceinline__ int slot_owner(int s, int Q, int R) {
  return s < R * (Q + 1) ? s / (Q + 1) : R + (s - R * (Q + 1)) / Q;
}

__device__ __forceinline__ float warp_max(float x) {  // NaN only if every lane has one
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Sums each of G values over the warp: a lane ends with one head's sum in l[0], and returns which.
template <int G>
__device__ __forceinline__ int head_sums(float (&l)[G], int lane) {
  int h = 0, o = 16;
#pragma unroll
  for (int n = G / 2; n > 0; n >>= 1, o >>= 1) {  // half of the heads go to the other half of the lanes
    const bool up = lane & o;
    h += up ? n : 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? l[i + n] : l[i], give = up ? l[i] : l[i + n];
      l[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
  return h;
}
// Two halves to two e4m3 codes, and back (exact).
__device__ __forceinline__ uint32_t e4m3x2_half(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
  return r;
}
__device__ __forceinline__ __half2 half_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return *reinterpret_cast<const __half2 *>(&h);
}
__device__ __forceinline__ float fin(float m) { return m == -INFINITY ? 0.f : m; }
// vs: the V scales of a warp's tiles, one a lane, whose 4096 bytes of codes (of block blk) are at rows +
// blk * block_bytes.  A block of zeros has the scale 1, which says nothing of its size, and would let
// its keys set the reference of a tile whose other blocks are small: where the codes are zeros (and
// NaNs, which come out whatever their weight is) alone, the scale becomes the least there is.  Looked at
// only where a scale is 1, and a block that is not zeros mostly shows it in its first 16 codes: 512
// units of 1100 rows take 31 us with or without scales of 1, 49 us when all of V is zeros.
__device__ __forceinline__ bool zero_codes(const uint4 *at) {
  const uint4 x = __ldcg(at);
  // a magnitude m that is neither 0 nor 127 leaves a bit of m + 1 between the lowest and the highest
  return ((((x.x & 0x7f7f7f7fu) + 0x01010101u) | ((x.y & 0x7f7f7f7fu) + 0x01010101u) |
           ((x.z & 0x7f7f7f7fu) + 0x01010101u) | ((x.w & 0x7f7f7f7fu) + 0x01010101u)) & 0x7e7e7e7eu) == 0;
}
__device__ __noinline__ float without_zeros(const uint8_t *rows, int block_bytes, int blk, float vs, int lane) {
  const uint8_t *mine = rows + (size_t)blk * block_bytes;
  uint32_t todo = __ballot_sync(0xffffffffu, vs == 1.f && zero_codes(reinterpret_cast<const uint4 *>(mine)));
#pragma unroll 1
  for (; todo != 0; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const uint4 *at = reinterpret_cast<const uint4 *>(rows + (size_t)__shfl_sync(0xffffffffu, blk, src) * block_bytes);
    bool zero = true;
#pragma unroll 2  // few registers: the softmax warps keep theirs over the call
    for (int i = 0; i < 8; ++i) zero &= zero_codes(at + lane + 32 * i);
    if (__all_sync(0xffffffffu, zero) && lane == src) vs = 0x1p-126f;
  }
  return vs;
}
// 2^(m - to), the factor of a sum kept relative to m (-inf: an empty one, or NaN, which stays)
__device__ __forceinline__ float rescale(float m, float to) { return m == -INFINITY ? 0.f : ex2(m - to); }

// A stage of the ring and the parity of its use: K's stages are the even ones, V's the odd.
template <int NST>
struct StageOf {
  int st;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    st += 2;
    if (st >= NST) {
      st -= NST;
      ph ^= 1;
    }
  }
  __device__ __forceinline__ StageOf before() const {  // the one before this one
    StageOf p = *this;
    p.st -= 2;
    if (p.st < 0) {
      p.st += NST;
      p.ph ^= 1;
    }
    return p;
  }
};

// A CTA's share of one unit.
struct Seg {
  int u, n0;          // rows before the append
  int lo, t8, b_hi;   // 8-bit blocks [lo, b_hi) in t8 tiles
  int tail_old, nt;   // tail rows before and after the append, if this share has the tail (else nt = 0)
  bool tail, add;     // has the unit's last slot; appends
  bool whole;         // is the whole unit
  int ntiles;
};

// The maps of K's and V's codes, in boxes of a tile and of a block, of their tails, and of the rows
// of the block completed last.
struct Maps {
  CUtensorMap k, v, k1, v1, kt, vt, kl, vl;
};

// One shared unit: its segments' results are at part(0), part(1), ...
struct Shared {
  int u, nseg, first, next;  // slots: first, then next, next + 2, ...
  __device__ __forceinline__ int slot(int s) const { return s == 0 ? first : next + 2 * (s - 1); }
};

__device__ __forceinline__ float seg_weight(float2 ml, float m) {
  return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - m);  // empty: 0; NaN stays
}
__device__ __forceinline__ uint2 bf4(float4 o, float inv) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Looks at the CTA's marked units, by all warps: the mark stays with those whose open rows are in kl and
// vl; rows that are gone are reported.  (Another CTA that has planned may already have written to a
// unit's tail; only the CTA that has the tail goes by the mark.)
template <int D>
__device__ __noinline__ void check_marks(const P8 &p, int *marks, const int *sn, int u_first, int nu, int warp,
                                         int lane) {
  constexpr int RV = D / 8;
#pragma unroll 1
  for (int i = warp; i < nu; i += NWARP) {
    const int u = u_first + i, n = i < SNAP ? sn[i] : ~p.snap[u];
    if (i < SNAP ? ((marks[1 + i / 32] >> (i % 32)) & 1) == 0 : n < 0) continue;
    const int open = open_rows(n, p.c.blocks[u]);
    bool left = true;  // the tail's first row is the one that the last call left
    if (lane < 2 * RV) {
      const uint4 *tl = reinterpret_cast<const uint4 *>(lane < RV ? p.c.kt : p.c.vt) + (size_t)u * KB8 * RV;
      const uint4 *ls = reinterpret_cast<const uint4 *>(lane < RV ? p.c.kl : p.c.vl) + ((size_t)u * KL8 + KB8) * RV;
      left = same16(__ldcg(tl + lane % RV), __ldcg(ls + lane % RV));
    }
    left = __all_sync(0xffffffffu, left);
    if (lane == 0 && !(left && open == OPEN_LAST)) {
      if (left && open == OPEN_GONE) set_status(p.status, KVC_DEV_BAD_STATE);
      if (i < SNAP) atomicAnd(marks + 1 + i / 32, ~(1 << (i % 32)));
      else p.snap[u] = n;
    }
  }
}

// The new row is the first of a block, or joins rows that are kept: the kept ones go back to the tail,
// unless the block is then complete.  By a warp.  (What is written here concerns the unit's open rows,
// so it misleads no CTA but the one that has them, which has planned.)
template <int D>
__device__ __noinline__ void open_block(const P8 &p, int u, int n0, int lane) {
  constexpr int RV = D / 8;
  const int r = n0 % KB8;
  if (r == KB8 - 1) return;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint4 *tail = reinterpret_cast<uint4 *>(h ? p.c.vt : p.c.kt) + (size_t)u * KB8 * RV;
    uint4 *kept = reinterpret_cast<uint4 *>(h ? p.c.vl : p.c.kl) + (size_t)u * KL8 * RV;
#pragma unroll 8
    for (int e = lane; e < r * RV; e += 32) tail[e] = __ldcg(kept + e);
    const uint4 *first = r > 0 ? kept : reinterpret_cast<const uint4 *>(h ? p.v_new : p.k_new) + (size_t)u * RV;
    if (lane < RV) kept[KB8 * RV + lane] = __ldcg(first + lane);
  }
  if (lane == 0 && (r > 0 || p.c.blocks[u].x != n0 / KB8)) p.c.blocks[u] = make_int2(n0 / KB8, -1);
}

// Quantises unit u's block nb, which the new row completes, and keeps its rows as they came, by the
// 128 output threads; re: the other rows are the kept ones.
template <int D>
__device__ __noinline__ void complete(const P8 &p, int u, int nb, bool re, uint32_t *red, int t) {
  constexpr int RV = D / 8, NP = KB8 * RV / KV8_NT, RS = KV8_NT / RV;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const uint4 *xn = reinterpret_cast<const uint4 *>(h ? p.v_new : p.k_new) + (size_t)u * RV;
    uint4 *kept = reinterpret_cast<uint4 *>(h ? p.c.vl : p.c.kl) + (size_t)u * KL8 * RV;
    const uint4 *old = re ? kept : reinterpret_cast<const uint4 *>(h ? p.c.vt : p.c.kt) + (size_t)u * KB8 * RV;
    uint4 w[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) w[i] = t / RV + i * RS < KB8 - 1 ? old[t + i * KV8_NT] : xn[t % RV];
    if (p.c.blocks) {
#pragma unroll
      for (int i = 0; i < NP; ++i) kept[t + i * KV8_NT] = w[i];
      if (!re && t < RV) kept[KB8 * RV + t] = w[0];  // the tail's first row is this block's
      if (h == 0 && t == 0) p.c.blocks[u] = make_int2(nb + 1, nb);
    }
    quantise_block<D>(w, (h ? p.c.vq : p.c.kq) + ((size_t)u * p.c.cap + (size_t)nb * KB8) * D,
                      (h ? p.c.vs : p.c.ks) + (size_t)u * (p.c.cap / KB8) + nb, red, 3, t);
  }
}

// Merges a shared unit's few segments (at most FEW) by nt threads, t of them this one.
template <int D, int G>
__device__ __noinline__ void merge_few(const float2 *part_ml, const float *part_o, __nv_bfloat16 *out, int ga,
                                       Shared x, int t, int nt) {
#pragma unroll 1
  for (int i = t; i < ga * (D / 4); i += nt) {
    const int h = i / (D / 4), c = i % (D / 4);
    float2 ml[FEW];
    float4 o[FEW];
#pragma unroll
    for (int s = 0; s < FEW; ++s)
      if (s < x.nseg) {
        ml[s] = __ldcg(part_ml + x.slot(s) * G + h);
        o[s] = __ldcg(reinterpret_cast<const float4 *>(part_o + ((size_t)x.slot(s) * G + h) * D) + c);
      }
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < FEW; ++s)
      if (s < x.nseg) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int s = 0; s < FEW; ++s)
      if (s < x.nseg) {
        const float w = seg_weight(ml[s], m);
        l += ml[s].y * w;
        a.x += o[s].x * w, a.y += o[s].y * w, a.z += o[s].z * w, a.w += o[s].w * w;
      }
    reinterpret_cast<uint2 *>(out + ((size_t)x.u * ga + h) * D)[c] = bf4(a, 1.f / l);
  }
}

// Merges a shared unit's segments by the whole CTA; buf: shared memory.
template <int D, int G>
__device__ __forceinline__ void merge_cta(const P8 &p, const Shared &x, float *buf, int tid) {
  constexpr int NT = 512, NI = G * D / 4, NG = NT / NI;  // four outputs a thread, NG groups of segments
  static_assert(NG >= 1, "threads");
  float2 *ml = reinterpret_cast<float2 *>(buf);             // [MAXCTA][G]
  float *w = buf + 2 * MAXCTA * G, *inv = w + MAXCTA * G;   // [MAXCTA][G], [G]
  float4 *acc = reinterpret_cast<float4 *>(inv + 8);        // [NT]
  for (int i = tid; i < x.nseg * G; i += NTH) ml[i] = __ldcg(p.part_ml + x.slot(i / G) * G + i % G);
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  if (warp < G) {
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < x.nseg; s += 32) m = fmaxf(m, ml[s * G + warp].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int s = lane; s < x.nseg; s += 32) {
      const float2 v = ml[s * G + warp];
      const float f = seg_weight(v, m);
      w[s * G + warp] = f;
      l += v.y * f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) inv[warp] = 1.f / l;
  }
  __syncthreads();
  const int i = tid % NI, h = i / (D / 4), c = i % (D / 4);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = tid < NT ? tid / NI : x.nseg; s < x.nseg; s += NG) {
    const float4 o = __ldcg(reinterpret_cast<const float4 *>(p.part_o + ((size_t)x.slot(s) * G + h) * D) + c);
    const float f = w[s * G + h];
    a.x += o.x * f, a.y += o.y * f, a.z += o.z * f, a.w += o.w * f;
  }
  if (tid < NT) acc[tid] = a;
  __syncthreads();
  if (tid < NI && h < p.ga) {
#pragma unroll
    for (int j = 1; j < NG; ++j) {
      const float4 o = acc[tid + j * NI];
      a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
    }
    reinterpret_cast<uint2 *>(p.out + ((size_t)x.u * p.ga + h) * D)[c] = bf4(a, inv[h]);
  }
  __syncthreads();
}

template <int D, int G>
__global__ void __launch_bounds__(NTH, 1)
    kv8_decode_kernel(const __grid_constant__ Maps maps, const __grid_constant__ P8 p) {
  using Gm = Geo<D, G>;
  constexpr int HB = Gm::HB, KPR = Gm::KPR, TB = Gm::TB, PN = Gm::PN, NST = Gm::NST;
  using Stage = StageOf<NST>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem), bar = sb + Gm::OFF_BAR;
  volatile int *misc = reinterpret_cast<volatile int *>(smem + Gm::OFF_BAR + B_MISC);
  int *sn = reinterpret_cast<int *>(smem + Gm::OFF_SN);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Wait wait{reinterpret_cast<WaitState *>(smem + Gm::OFF_BAR + B_MISC + 4 * M_WAIT)};
  const int U = p.c.units, cap = p.c.cap, b = blockIdx.x;
  const bool app = p.k_new != nullptr;

  for (int e = tid; e < (2 * QN * D * 3) / 16; e += NTH)  // unused query rows stay zero
    reinterpret_cast<uint4 *>(smem + Gm::OFF_Q8)[e] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (tid == 0) {
    *wait.s = {0, p.status, p.timeout};
    misc[M_UF] = misc[M_PF] = 0;
    misc[M_UL] = -1;
    misc[M_PL] = 0;
    misc[M_TODO + 1] = misc[M_TODO + 5] = 0;
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar + B_FULL + 8 * i, 1);
      mbar_init(bar + B_EMPTY + 8 * i, 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(bar + B_SFULL + 8 * i, 1);
      mbar_init(bar + B_SEMPTY + 8 * i, 4);
      mbar_init(bar + B_PFULL + 8 * i, 4);
      mbar_init(bar + B_OFULL + 8 * i, 1);
      mbar_init(bar + B_OEMPTY + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B_QFULL + 8 * i, 1);
      mbar_init(bar + B_QEMPTY + 8 * i, 1);
      mbar_init(bar + B_RFULL + 8 * i, 8);
      mbar_init(bar + B_REMPTY + 8 * i, 4);
    }
    mbar_init(bar + B_START, 11);  // W_S, W_PV, W_Q and the softmax warps
    fence_mbar_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.kt);
    tma_prefetch_desc(&maps.vt);
  }
  if (warp == W_M && lane <= SNAP / 32) misc[M_RE + lane] = 0;
  if (warp == W_S) {
    tmem_alloc(smem_u32(const_cast<int *>(misc + M_TMEM)), TMEM_COLS);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------- plan -------------------------------
  auto clamped = [&](int n) { return n < 0 ? 0 : min(n, cap); };
  const int per = (U + NTH - 1) / NTH;
  const int ua = min(U, tid * per), ub = min(U, ua + per);
  int sum = 0, n_own = 0;  // n_own: the row count of this thread's unit where it has only one
  int open_own = OPEN_TAIL;  // and where that one's open rows are
  constexpr int TW = TB * (HB / 4);  // slots of a tail and a unit's end: about a tile's time, two with 8 heads
  uint32_t odd = 0;
#pragma unroll 4
  for (int u = ua; u < ub; ++u) {
    const int n = p.c.n_valid[u];
    const int2 blk = per == 1 && p.c.blocks ? p.c.blocks[u] : make_int2(-1, -1);
    n_own = clamped(n);
    open_own = open_rows(n_own, blk);
    sum += n_own / KB8 + TW;
    odd |= n != n_own ? KVC_DEV_BAD_STATE : (app && n == cap ? KVC_DEV_CACHE_FULL : 0u);
  }
  if (b == 0 && odd) set_status(p.status, odd);
  auto rows_of = [&](int u) { return per == 1 ? n_own : clamped(p.c.n_valid[u]); };  // u: own
  // Sums over the CTA, one barrier each; two sets of shared words in turn, so that a warp that
  // writes one has seen every warp done with it.  (The plan runs once, and so at the rate at
  // which its instructions are fetched: 2.1 us for 8 units with two scans and
  // atomic counts, 1.5 so.)
  int set = 0;
  auto warp_sums = [&](int x, int lanes) {  // x: a warp's; the sum of the first `lanes` warps'
    volatile int *w = misc + M_WS + set * NWARP;
    set ^= 1;
    if (lane == 31) w[warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < lanes ? w[lane] : 0);
  };
  tc_fence_before();
  const int total = warp_sums(__reduce_add_sync(0xffffffffu, sum), NWARP);
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform(misc[M_TMEM]);
  const int P = min((int)gridDim.x, (total + MINS - 1) / MINS);
  const int Q = total / P, R = total - Q * P;
  // Few units: shares of up to C slots that each lie in one unit, where that costs little
  // against the even split (a share that crosses units has two results to merge).
  int C = 0, shares = 0;
  auto shares_of = [&](int c) { return ua < ub ? (sum - TW) / c + 1 : 0; };  // of this thread's one unit
  if (U <= (int)gridDim.x) {
    const int even = (total + (int)gridDim.x - 1) / (int)gridDim.x, most = max(MINC, even + 6 + even / 16);
    int c = max(MINC, even);
#pragma unroll 1
    for (int i = 0; i < 8 && c <= most; ++i) {
      shares = warp_sums(__reduce_add_sync(0xffffffffu, shares_of(c)), NWARP);
      if (shares <= (int)gridDim.x) {
        C = c;
        break;
      }
      c += max(1, c / 16);
    }
  }
  // before this thread's units: shares of size C, or slots
  const int mine = C > 0 ? shares_of(C) : sum;
  int pre = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += t;
  }
  pre += warp_sums(pre, warp) - mine;
  int s0, s1;
  if (C > 0) {
    if (pre <= b && b < pre + mine) misc[M_UF] = misc[M_UL] = ua, misc[M_PF] = misc[M_PL] = pre;
    s0 = b < shares ? 0 : 1;
    s1 = 1;
  } else {
    s0 = slot_first(min(b, P), Q, R);
    s1 = slot_first(min(b + 1, P), Q, R);
    if (s0 < s1 && ((pre <= s0 && s0 < pre + sum) || (pre < s1 && s1 <= pre + sum))) {
      int at = pre;
#pragma unroll 1
      for (int u = ua; u < ub; ++u) {
        const int nb = rows_of(u) / KB8, nx = at + nb + TW;
        if (at <= s0 && s0 < nx) {  // the tail is its first slot's; who begins behind that has none of u
          const bool past = s0 > at + nb;
          misc[M_UF] = past ? u + 1 : u, misc[M_PF] = past ? nx : at;
        }
        if (at < s1 && s1 <= nx) misc[M_UL] = u, misc[M_PL] = at;
        at = nx;
      }
    }
  }
  __syncthreads();
  const int u_first = uniform(misc[M_UF]), p_first = uniform(misc[M_PF]), u_last = uniform(misc[M_UL]),
            p_last = uniform(misc[M_PL]);
  const int nu = s0 < s1 ? max(u_last - u_first + 1, 0) : 0;
#pragma unroll 1
  for (int i = per > 1 ? tid : (ua < ub && ua >= u_first ? ua - u_first : nu); i < nu; i += NTH) {
    const int u = u_first + i;
    int n = n_own, open = open_own;
    if (per > 1) {
      n = clamped(p.c.n_valid[u]);
      open = p.c.blocks ? open_rows(n, p.c.blocks[u]) : OPEN_TAIL;
    }
    if (open != OPEN_TAIL) {
      misc[M_RE] = 1;
      if (i < SNAP) atomicOr(const_cast<int *>(misc) + M_RE + 1 + i / 32, 1 << (i % 32));
      else n = ~n;
    }
    if (i < SNAP) sn[i] = n;
    else p.snap[u] = n;
  }
  __syncthreads();
  if (misc[M_RE]) {  // rarely: a row count was lowered
    check_marks<D>(p, const_cast<int *>(misc) + M_RE, sn, u_first, nu, warp, lane);
    __syncthreads();
  }
  // The slots at which its first unit's share begins and its last one's ends, within the unit.  (By
  // way of a shuffle, for the compiler would compute them again wherever they are used.)
  const int lo_first = uniform(C > 0 ? (b - p_first) * C : max(s0 - p_first, 0));
  const int hi_last = uniform(C > 0 ? lo_first + C : s1 - p_last);
  // The CTA's k-th unit: the last one first.
  auto seg_at = [&](int k) {
    const int i = k == 0 ? nu - 1 : k - 1;
    Seg g;
    g.u = u_first + i;
    g.n0 = i < SNAP ? sn[i] : max(p.snap[g.u], ~p.snap[g.u]);
    g.add = app && g.n0 < cap;
    const int nb = g.n0 / KB8;
    g.lo = i == 0 ? lo_first : 0;
    const int hi = i == nu - 1 ? hi_last : nb + TW;
    g.tail = hi > nb;
    g.whole = g.lo == 0 && g.tail;
    g.b_hi = min(hi, nb);
    g.t8 = g.b_hi > g.lo ? (g.b_hi - g.lo + TB - 1) / TB : 0;
    g.tail_old = g.n0 - nb * KB8;
    g.nt = g.tail ? g.tail_old + (g.add ? 1 : 0) : 0;
    g.ntiles = g.t8 + (g.nt > 0 ? 1 : 0);
    return g;
  };
  // Whether unit u's open rows are in kl and vl.
  auto kept_rows = [&](int u) {
    if (misc[M_RE] == 0) return false;
    const int i = u - u_first;
    return i < SNAP ? ((misc[M_RE + 1 + i / 32] >> (i % 32)) & 1) != 0 : p.snap[u] < 0;
  };
  auto shared_at = [&](const Seg &g) {
    Shared x;
    x.u = g.u;
    const int nb = g.n0 / KB8;  // the tail's slot, which the last share has
    if (C > 0) {
      x.nseg = nb / C + 1;
      x.first = 2 * p_first;
      x.next = x.first + 2;
    } else {
      const int base = g.u == u_first ? p_first : p_last;
      const int b0 = slot_owner(base, Q, R);
      x.nseg = slot_owner(base + nb, Q, R) - b0 + 1;
      // the first segment may be its CTA's second result; the others are their CTA's first
      x.first = 2 * b0 + (slot_first(b0, Q, R) == base ? 0 : 1);
      x.next = 2 * (b0 + 1);
    }
    return x;
  };

  // one arrival a warp on B_START, once the loaded word x is there
  auto arrived = [&](uint32_t x) {
    if (__any_sync(0xffffffffu, x == 0xdeadbeefu)) __nanosleep(0);  // wants x, whatever it is
    if (lane == 0) mbar_arrive(bar + B_START);
  };
  // the same, for a converged warp whose lanes agree
  auto seg_uni = [&](int k) {
    Seg g = seg_at(k);
    g.u = uniform(g.u), g.n0 = uniform(g.n0), g.lo = uniform(g.lo), g.t8 = uniform(g.t8);
    g.b_hi = uniform(g.b_hi), g.tail_old = uniform(g.tail_old), g.nt = uniform(g.nt);
    g.ntiles = uniform(g.ntiles);
    return g;
  };
  if (warp == W_TMA) {
    {
      const uint32_t lead = elect_one();
      Stage k8{0}, v8{1};
      int tiles = 0;
      bool ok = true;
      for (int k = 0; k < nu && ok; ++k) {
        const Seg g = seg_uni(k);
        int row = (g.u * (cap / KB8) + g.lo) * Gm::BR;
        for (int i = 0; i < g.ntiles; ++i, ++tiles, row += TROWS) {
          // Small loads can wait microseconds behind the tiles of 152 SMs, so the flood begins
          // when the first unit's have come.
          if (tiles == 1 && !wait.all(bar + B_START, 0)) { ok = false; break; }
          const int nblk = min(TB, g.b_hi - g.lo - TB * i), boxes = (g.tail_old + 15) / 16;
          const bool kept = i >= g.t8 && kept_rows(g.u);
          const int open_row = g.u * (kept ? KL8 : KB8);
          auto load = [&](Stage &x, const CUtensorMap *whole, const CUtensorMap *one, const CUtensorMap *tail) {
            if (!wait.all(bar + B_EMPTY + 8 * x.st, x.ph ^ 1)) return false;
            const uint32_t dst = sb + x.st * SB, full = bar + B_FULL + 8 * x.st;
            if (i < g.t8) {
              expect_tx(lead, full, nblk * KB8 * D);
              if (nblk == TB) {
                tma_load(lead, dst, whole, 0, row, full);
              } else {
#pragma unroll 1
                for (int j = 0; j < nblk; ++j) tma_load(lead, dst + j * KB8 * D, one, 0, row + j * Gm::BR, full);
              }
            } else {  // 16 rows a box; the new row comes from k_new and v_new
              expect_tx(lead, full, boxes * Gm::KBT * 2048);
#pragma unroll 1
              for (int kb = 0; kb < Gm::KBT; ++kb)
#pragma unroll 1
                for (int j = 0; j < boxes; ++j)
                  tma_load(lead, dst + kb * KB8 * 128 + j * 2048, tail, kb * 64, open_row + j * 16, full);
            }
            x.next();
            return true;
          };
          if (!load(k8, &maps.k, &maps.k1, kept ? &maps.kl : &maps.kt) ||
              !load(v8, &maps.v, &maps.v1, kept ? &maps.vl : &maps.vt)) {
            ok = false;
            break;
          }
        }
      }
      // drain: every load issued has arrived before the CTA may exit (the last use of each stage)
#pragma unroll 1
      for (int j = 0; j < NST / 2; ++j) {
        k8 = k8.before();
        v8 = v8.before();
        if (j < tiles || !ok) {
          wait_drain(bar + B_FULL + 8 * k8.st, k8.ph, ok ? p.timeout : 0);
          wait_drain(bar + B_FULL + 8 * v8.st, v8.ph, ok ? p.timeout : 0);
        }
      }
    }
  } else if (warp == W_S) {
    const uint32_t lead = elect_one();
    Stage k8{0};
    int sc = 0, ka = 0;
    bool ok = true;
    // the appended row's pieces are loaded a unit ahead
    auto new_row = [&](int k) {
      return app && k < nu && lane < D / 8
                 ? *reinterpret_cast<const uint4 *>(p.k_new + (size_t)seg_at(k).u * D + lane * 8)
                 : make_uint4(0, 0, 0, 0);
    };
    uint4 xnext = new_row(0);
    arrived(xnext.x);
    for (int k = 0; k < nu && ok; ++k) {
      const Seg g = seg_uni(k);
      const uint4 xnew = xnext;
      xnext = new_row(k + 1);
      if (g.ntiles == 0) continue;
      const int qb = ka & 1;
      ok = wait.all(bar + B_QFULL + 8 * qb, (ka >> 1) & 1);
      for (int i = 0; i < g.ntiles && ok; ++i, k8.next(), ++sc) {
        const int st = k8.st, s = sc % NB;
        ok = wait.all(bar + B_FULL + 8 * st, k8.ph) && wait.all(bar + B_SEMPTY + 8 * s, ((sc / NB) & 1) ^ 1);
        if (!ok) break;
        uint8_t *tile = smem + st * SB;
        if (i >= g.t8 && g.add) {  // the appended row joins the tail's tile
          const int r = g.tail_old;
          if (lane < D / 8) {
            *reinterpret_cast<uint4 *>(tile + (lane >> 3) * KB8 * 128 + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = xnew;
            if (r < KB8 - 1)  // and the tail itself, unless it completes a block
              *reinterpret_cast<uint4 *>(p.c.kt + ((size_t)g.u * KB8 + r) * D + lane * 8) = xnew;
          }
          if (lane == 0 && p.c.pos) p.c.pos[(size_t)g.u * cap + g.n0] = p.new_pos;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        tc_fence_after();
        {
          const uint32_t d = tmem + T_S + s * 32;
          const uint64_t a = sdesc(sb + st * SB, 16, 1024, L_128B);
          if (i < g.t8) {
            const uint64_t q = sdesc(sb + Gm::OFF_Q8 + qb * QN * D, 16, 8 * D, D == 128 ? L_128B : L_64B);
#pragma unroll
            for (int j = 0; j < KPR; ++j)  // D = 64: the rows' first keys, then their second
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8(lead, d + j * QN, a + (j * D + kk * 32) / 16, q + 2 * kk, idesc8(QN, false), kk != 0);
          } else {
            const uint64_t q = sdesc(sb + Gm::OFF_QT + qb * QN * D * 2, 16, 1024, L_128B);
#pragma unroll
            for (int kb = 0; kb < Gm::KBT; ++kb)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16(lead, d, a + ((kb * KB8 * 128 + kk * 32) >> 4), q + ((kb * QN * 128 + kk * 32) >> 4),
                          idesc16(QN, false), (kb | kk) != 0);
          }
          mma_commit(lead, bar + B_SFULL + 8 * s);  // the softmax warps then free K's stage
          if (i == g.ntiles - 1) mma_commit(lead, bar + B_QEMPTY + 8 * qb);
        }
        __syncwarp();
      }
      if (ok) ++ka;
    }
    // every commit has arrived before the CTA may exit
    if (ka > 0) wait_drain(bar + B_QEMPTY + 8 * ((ka - 1) & 1), ((ka - 1) >> 1) & 1, p.timeout);
    if (!ok && sc > 0) wait_drain(bar + B_SFULL + 8 * ((sc - 1) % NB), ((sc - 1) / NB) & 1, p.timeout);
  } else if (warp == W_PV) {
    const uint32_t lead = elect_one();
    Stage v8{1};
    int sc = 0;
    bool ok = true;
    auto new_row = [&](int k) {
      return app && k < nu && lane < D / 8
                 ? *reinterpret_cast<const uint4 *>(p.v_new + (size_t)seg_at(k).u * D + lane * 8)
                 : make_uint4(0, 0, 0, 0);
    };
    uint4 xnext = new_row(0);
    arrived(xnext.x);
    for (int k = 0; k < nu && ok; ++k) {
      const Seg g = seg_uni(k);
      const uint4 xnew = xnext;
      xnext = new_row(k + 1);
      for (int i = 0; i < g.ntiles && ok; ++i, v8.next(), ++sc) {
        const int st = v8.st, s = sc % NB;
        ok = wait.all(bar + B_FULL + 8 * st, v8.ph);
        if (!ok) break;
        uint8_t *tile = smem + st * SB;
        const bool tail = i >= g.t8;
        if (tail && (g.add || (g.nt & 15))) {
          // the appended row, and zeros up to the next 16 (weights there are zero, but what
          // the buffer holds may be anything)
          auto at = [&](int r, int c) {
            return reinterpret_cast<uint4 *>(tile + (c >> 3) * KB8 * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          };
          if (g.add && lane < D / 8) {
            *at(g.tail_old, lane) = xnew;
            if (g.tail_old < KB8 - 1)
              *reinterpret_cast<uint4 *>(p.c.vt + ((size_t)g.u * KB8 + g.tail_old) * D + lane * 8) = xnew;
          }
          const int r1 = (g.nt + 15) & ~15;
#pragma unroll 1
          for (int e = lane; e < (r1 - g.nt) * (D / 8); e += 32)
            *at(g.nt + e / (D / 8), e % (D / 8)) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        ok = wait.all(bar + B_PFULL + 8 * s, (sc / NB) & 1);
        if (!ok) break;
        tc_fence_after();
        {
          const uint32_t d = tmem + T_O + s * 64, va = sb + st * SB, pa = sb + Gm::OFF_P + s * Gm::PB;
          if (!tail) {
            // 32 rows a step.  D = 64: lanes 0-63 hold the rows' first keys' columns of V, 64-127
            // their second's, and so do the two halves of the weights' columns: each half of the
            // lanes has its keys' sums in its half of the columns
            const uint64_t a = sdesc(va, 0, 1024, L_128B), w = sdesc(pa, 128, TROWS * 16, L_NONE);
            const int steps = min(TB, g.b_hi - g.lo - TB * i) * Gm::BR / 32;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f8(ks < steps ? lead : 0u, d, a + ks * (4096 / 16), w + ks * (512 / 16), idesc8(KPR * PN, true),
                     ks != 0);
          } else {
            const int steps = (g.nt + 15) / 16;
#pragma unroll 1
            for (int ks = 0; ks < steps; ++ks)  // D = 64: both halves of the lanes read the same columns
              mma_bf16(lead, d, sdesc(va + ks * 2048, D == 128 ? KB8 * 128 : 0, 1024, L_128B),
                        sdesc(pa + ks * 256, 128, KB8 * 16, L_NONE), idesc16(16, true), ks != 0);
          }
          mma_commit(lead, bar + B_OFULL + 8 * s);  // the output warps then free V's stage
        }
        __syncwarp();
      }
    }
    if (sc > 0)  // the last commit has arrived before the CTA may exit
      wait_drain(bar + B_OFULL + 8 * ((sc - 1) % NB), ((sc - 1) / NB) & 1, p.timeout);
  } else if (warp == W_Q) {
    // ---------------- queries: two e4m3 terms, and bf16 for the tail ----------------
    // Two operands (the S warp's commit frees one), but eight sets of factors: the softmax
    // warps may be NB tiles behind the S product, and unit ka + 8 is written once the product
    // of unit ka + 6's last tile is done, six or more tiles after unit ka's last.
    // A lane holds E columns of one head: LPH lanes a head, so all heads' steps are one.
    constexpr int LPH = 32 / G, E = D / LPH;
    float *qs = reinterpret_cast<float *>(smem + Gm::OFF_QS);
    const int h = lane / LPH, c0 = (lane % LPH) * E;
    int ka = 0;
    bool ok = true;
    auto write_q = [&](int k) {
      const Seg g = seg_at(k);
      if (g.ntiles == 0) return;
      const int qb = ka & 1;
      uint32_t w[E / 2];
      const __nv_bfloat16 *src = p.q + ((size_t)g.u * p.ga + h) * D + c0;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) w[e] = 0;
      if (h < p.ga) {
        if (E == 2) w[0] = *reinterpret_cast<const uint32_t *>(src);
        else if (E == 4) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(src);
        else
#pragma unroll
          for (int e = 0; e < E / 8; ++e)
            reinterpret_cast<uint4 *>(w)[e] = reinterpret_cast<const uint4 *>(src)[e];
      }
      if (ka >= 2) ok = wait.all(bar + B_QEMPTY + 8 * qb, ((ka - 2) >> 1) & 1);
      if (!ok) return;
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int ex = kv8_exponent(m);
      // a head with an infinity or a NaN in it has only NaN terms, and so only NaN logits
      const float inv = m >= 0x7f80u ? __uint_as_float(0x7fc00000u) : exp2_int(-ex);
      if (c0 == 0) qs[(ka & 7) * 8 + h] = exp2_int(ex) * p.lc;  // see the softmax warps
      uint32_t t[2][(E + 3) / 4];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float a = bf_lo(w[e]) * inv, c = bf_hi(w[e]) * inv;
        const uint32_t hi = e4m3x2(a, c);
        const float2 f = e4m3x2_float(hi);
        const uint32_t lo = e4m3x2((a - f.x) * 16.f, (c - f.y) * 16.f);
        t[0][e / 2] = e % 2 ? t[0][e / 2] | (hi << 16) : hi;
        t[1][e / 2] = e % 2 ? t[1][e / 2] | (lo << 16) : lo;
      }
      uint8_t *q8 = smem + Gm::OFF_Q8 + qb * QN * D, *qt = smem + Gm::OFF_QT + qb * QN * D * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = j * HB + h, sw = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
        for (int e = 0; e < (E + 15) / 16; ++e) {
          uint8_t *d = q8 + r * D + ((((c0 >> 4) + e) ^ sw) << 4) + (c0 & 15);
          if (E == 2) *reinterpret_cast<uint16_t *>(d) = (uint16_t)t[j][0];
          else if (E == 4) *reinterpret_cast<uint32_t *>(d) = t[j][0];
          else if (E == 8) *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<uint2 *>(t[j]);
          else *reinterpret_cast<uint4 *>(d) = reinterpret_cast<uint4 *>(t[j])[e];
        }
      }
#pragma unroll
      for (int e = 0; e < (E + 7) / 8; ++e) {
        uint8_t *d = qt + (c0 >> 6) * QN * 128 + h * 128 + (((((c0 & 63) >> 3) + e) ^ (h & 7)) << 4) + (c0 & 7) * 2;
        if (E == 2) *reinterpret_cast<uint32_t *>(d) = w[0];
        else if (E == 4) *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<uint2 *>(w);
        else *reinterpret_cast<uint4 *>(d) = reinterpret_cast<uint4 *>(w)[e];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + B_QFULL + 8 * qb);
      ++ka;
    };
    if (nu > 0) write_q(0);
    if (lane == 0) mbar_arrive(bar + B_START);
    for (int k = 1; k < nu && ok; ++k) write_q(k);
    // then blocks that begin, and kept rows that go back to the tail: not before the queries, for the
    // softmax warps wait for those (1216 units of 544 rows, D = 64, 8 heads: 33.0 us; in write_q 41.5)
    if (app && p.c.blocks && ok)
#pragma unroll 1
      for (int k = 0; k < nu; ++k) {
        const Seg g = seg_at(k);
        if (g.tail && g.add && (g.tail_old == 0 || kept_rows(g.u))) open_block<D>(p, g.u, g.n0, lane);
      }
  } else if (warp < W_OUT) {
    // ------------------ softmax: two sets of four warps, alternate tiles ------------------
    const int set = (warp - W_SM) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    const float *qs = reinterpret_cast<const float *>(smem + Gm::OFF_QS);
    float *mx = reinterpret_cast<float *>(smem + Gm::OFF_MX) + set * 2 * 8 * 4;
    float *mt = reinterpret_cast<float *>(smem + Gm::OFF_MT);
    float2 *stat = reinterpret_cast<float2 *>(smem + Gm::OFF_ST);
    const int bo = KPR == 2 ? quarter : quarter >> 1;  // this warp's 32 rows lie in one block
    // The scales of the warp's next 32 tiles in a segment, one a lane, loaded long before their
    // use (a load can wait for microseconds behind the tiles): a segment's first ones while the
    // segment before is worked on.
    auto scales = [&](const Seg &g, int first, int chunk, float &ks, float &vs) {
      const int i = first + 2 * (chunk * 32 + lane), blk = g.lo + TB * i + bo;
      const bool in = i < g.t8 && blk < g.b_hi;
      const size_t at = (size_t)g.u * (cap / KB8) + blk;
      // (not by way of the read-only cache: the step before writes scales while this CTA may be resident)
      ks = in ? __ldcg(p.c.ks + at) : 1.f;
      vs = in ? __ldcg(p.c.vs + at) : 0.5f;  // not 1
    };
    int sc = 0, ka = 0;
    bool ok = true;  // after a wait ran out the warps still meet at every barrier
    Stage k8{0};
    float ksn = 1.f, vsn = 1.f;
    if (nu > 0) scales(seg_at(0), set, 0, ksn, vsn);
    arrived(__float_as_uint(ksn) ^ __float_as_uint(vsn));
    for (int k = 0; k < nu; ++k) {
      const Seg g = seg_uni(k);
      float ksl = ksn, vsl = vsn, ksl2 = 1.f, vsl2 = 1.f;
      if (k + 1 < nu) scales(seg_at(k + 1), (sc + g.ntiles + set) & 1, 0, ksn, vsn);
      if (g.ntiles == 0) continue;
      float m_run[G], l_run[G];
#pragma unroll
      for (int h = 0; h < G; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;
      const int first = (sc + set) & 1;
      for (int i = 0; i < g.ntiles; ++i, ++sc, k8.next()) {
        if ((sc & 1) != set) continue;
        const int par = (sc >> 1) & 1, own = (i - first) >> 1, buf = sc % NB, use = (sc / NB) & 1;
        const bool tail = i >= g.t8;
        if ((own & 31) == 0) {
          if (own > 0) ksl = ksl2, vsl = vsl2;
          if (__any_sync(0xffffffffu, vsl == 1.f))
            vsl = without_zeros(p.c.vq + (size_t)g.u * cap * D + (D == 128 ? (quarter & 1) * 4096 : 0), KB8 * D,
                                g.lo + TB * (first + 2 * (own + lane)) + bo, vsl, lane);
          if (g.t8 > 2 * (own + 32)) scales(g, first, own / 32 + 1, ksl2, vsl2);
        }
        const float ks = __shfl_sync(0xffffffffu, ksl, own & 31), vs = tail ? 1.f : __shfl_sync(0xffffffffu, vsl, own & 31);
        const bool have = tail ? row < g.nt : g.lo + TB * i + bo < g.b_hi;
        ok = ok && wait.all(bar + B_SFULL + 8 * buf, use);
        float s[KPR][HB], f[G];
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < G; ++h)  // kept off 0 and infinity, which times a masked row's are NaN
            f[h] = tail ? p.lc : fminf(fmaxf(qs[(ka & 7) * 8 + h] * ks, 1e-37f), 3e38f);
#pragma unroll
          for (int j = 0; j < KPR; ++j) {
            float r[2 * HB];
            if (HB == 4) tmem_ld8(tq + T_S + buf * 32 + j * QN, r);
            else tmem_ld16(tq + T_S + buf * 32 + j * QN, r);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < G; ++h)
              s[j][h] = !have || (j > 0 && tail) ? -INFINITY : (tail ? r[h] : fmaf(r[HB + h], 0.0625f, r[h]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar + B_SEMPTY + 8 * buf);
            if (quarter == 0) mbar_arrive(bar + B_EMPTY + 8 * k8.st);
          }
        }
        const float ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
        float wm[G];
        bool grew = false;
#pragma unroll
        for (int h = 0; h < G; ++h) wm[h] = warp_max(KPR == 2 ? fmaxf(s[0][h], s[KPR - 1][h]) : s[0][h]);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          wm[h] *= f[h];
          if (lane == 0) mx[(par * 8 + h) * 4 + quarter] = wm[h] + ev;
          grew |= wm[h] > m_run[h];
        }
        if (grew)  // the same in every lane
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mn = fmaxf(m_run[h], wm[h]);
            l_run[h] *= rescale(m_run[h], mn);
            m_run[h] = mn;
          }
        named_bar(1 + set, 128);  // every warp comes here, whatever its waits gave
        float x[KPR][HB], mkeep = 0.f;
        const float ev8 = tail ? ev : ev + 8.f;  // 256 times the weights: e4m3's upper range
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float4 m4 = *reinterpret_cast<const float4 *>(mx + (par * 8 + h) * 4);
          const float M = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), off = ev8 - fin(M);
#pragma unroll
          for (int j = 0; j < KPR; ++j) x[j][h] = ex2(fmaf(s[j][h], f[h], off));
          if (lane == h) mkeep = M;  // kept by lane h until the buffer is free
        }
#pragma unroll
        for (int h = G; h < HB; ++h)
#pragma unroll
          for (int j = 0; j < KPR; ++j) x[j][h] = 0.f;
        // the buffers' last tile has been read: its weights, its references and its product
        ok = ok && wait.all(bar + B_OEMPTY + 8 * buf, use ^ 1);
        if (!ok) continue;
        if (quarter == 0 && lane < G) mt[buf * 8 + lane] = mkeep;
        uint8_t *pb = smem + Gm::OFF_P + buf * Gm::PB + (row >> 3) * 128 + (row & 7) * 16;
        if (!tail) {
#pragma unroll
          for (int jj = 0; jj < KPR; ++jj) {
            // three e4m3 terms, a factor 16 apart, of each weight rounded to fp16 (2^-11; the
            // differences are exact there)
            uint32_t t[3][HB / 4];
            const __half2 x16 = __float2half2_rn(16.f);
#pragma unroll
            for (int w = 0; w < HB / 4; ++w) {
              __half2 a = __floats2half2_rn(x[jj][4 * w], x[jj][4 * w + 1]);
              __half2 c = __floats2half2_rn(x[jj][4 * w + 2], x[jj][4 * w + 3]);
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const uint32_t ca = e4m3x2_half(a), cc = e4m3x2_half(c);
                t[j][w] = ca | (cc << 16);
                if (j < 2) {
                  a = __hmul2(__hsub2(a, half_e4m3x2(ca)), x16);
                  c = __hmul2(__hsub2(c, half_e4m3x2(cc)), x16);
                }
              }
            }
            uint8_t *q = pb + jj * (PN / 16) * TROWS * 16;
            if (HB == 4) {
              *reinterpret_cast<uint4 *>(q) = make_uint4(t[0][0], t[1][0], t[2][0], 0);
            } else {
              *reinterpret_cast<uint4 *>(q) = make_uint4(t[0][0], t[0][HB / 4 - 1], t[1][0], t[1][HB / 4 - 1]);
              *reinterpret_cast<uint4 *>(q + TROWS * 16) = make_uint4(t[2][0], t[2][HB / 4 - 1], 0, 0);
            }
          }
        } else if (row < KB8) {
          uint32_t hi[HB / 2], lo[HB / 2];
#pragma unroll
          for (int w = 0; w < HB / 2; ++w) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x[0][2 * w], x[0][2 * w + 1]);
            hi[w] = *reinterpret_cast<const uint32_t *>(&a);
            const __nv_bfloat162 c = __floats2bfloat162_rn(x[0][2 * w] - bf_lo(hi[w]), x[0][2 * w + 1] - bf_hi(hi[w]));
            lo[w] = *reinterpret_cast<const uint32_t *>(&c);
          }
          if (HB == 4) {  // the second group's columns are not read
            *reinterpret_cast<uint4 *>(pb) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint4 *>(pb) = make_uint4(hi[0], hi[1], hi[HB / 2 - 2], hi[HB / 2 - 1]);
            *reinterpret_cast<uint4 *>(pb + KB8 * 16) = make_uint4(lo[0], lo[1], lo[HB / 2 - 2], lo[HB / 2 - 1]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + B_PFULL + 8 * buf);
        // the normaliser's terms, when nobody waits for this tile any more
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float mf = fin(m_run[h]);
          float e = ex2(fmaf(s[0][h], f[h], -mf));
          if (KPR == 2) e += ex2(fmaf(s[KPR - 1][h], f[h], -mf));
          l_run[h] += e;
        }
      }
      // the segment's normaliser: this warp's rows
      const int rb = ka & 1;
      if (ka >= 2) ok = ok && wait.all(bar + B_REMPTY + 8 * rb, ((ka - 2) >> 1) & 1);
      const int hl = head_sums<G>(l_run, lane);  // of this lane's head
      float mh = m_run[0];
#pragma unroll
      for (int h = 1; h < G; ++h) mh = hl == h ? m_run[h] : mh;
      if (ok && lane % (32 / G) == 0) stat[(rb * 8 + warp - W_SM) * 8 + hl] = make_float2(mh, l_run[0]);
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar + B_RFULL + 8 * rb);
      ++ka;
    }
  } else if (warp < W_M) {
    // ---------------- output: one head-dim lane a thread ----------------
    const int te = tid - 32 * W_OUT, quarter = warp & 3, d = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    const float *mtb = reinterpret_cast<const float *>(smem + Gm::OFF_MT);
    const float2 *stat = reinterpret_cast<const float2 *>(smem + Gm::OFF_ST);
    float *xh = reinterpret_cast<float *>(smem + Gm::OFF_X);
    float4 *mlb = reinterpret_cast<float4 *>(smem + Gm::OFF_ST + 2 * 8 * 8 * 8);  // [G] a segment's max, normaliser and its inverse
    constexpr uint32_t lanes = G >= 4 ? 0xffffffffu : (1u << (8 * (G & 3))) - 1;  // of a warp that has 8 G lanes
    if (app) {  // the last CTA to have planned advances the row counts
      if (te == 0) {
        __threadfence();
        misc[M_LAST] = atomicAdd(p.planned, 1) == (int)gridDim.x - 1;
      }
      named_bar(3, 128);
      if (misc[M_LAST]) {
        __threadfence();
#pragma unroll 4
        for (int u = te; u < U; u += 128) p.c.n_valid[u] = min(clamped(p.c.n_valid[u]) + 1, cap);
        if (te == 0) *p.planned = 0;
      }
      named_bar(3, 128);
    }
    Stage v8{1};
    int sc = 0, ka = 0, si = 0;
    bool ok = true;
    for (int k = 0; k < nu; ++k) {
      const Seg g = seg_at(k);
      float acc[G], M[G];
#pragma unroll
      for (int h = 0; h < G; ++h) acc[h] = 0.f, M[h] = -INFINITY;
      for (int i = 0; i < g.ntiles && ok; ++i, ++sc, v8.next()) {
        const int s = sc % NB;
        ok = wait.all(bar + B_PFULL + 8 * s, (sc / NB) & 1) && wait.all(bar + B_OFULL + 8 * s, (sc / NB) & 1);
        if (!ok) break;
        tc_fence_after();
        float o[PN], mtile[G];
        const uint32_t col = T_O + s * 64 + (D == 64 && quarter >= 2 ? PN : 0);
        if (PN == 16) tmem_ld16(tq + col, o);
        else tmem_ld32(tq + col, o);
#pragma unroll
        for (int h = 0; h < G; ++h) mtile[h] = mtb[s * 8 + h];
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar + B_OEMPTY + 8 * s);
          if (quarter == 0) mbar_arrive(bar + B_EMPTY + 8 * v8.st);
        }
        const bool tail = i >= g.t8;
        if (tail)  // a weight's second term may be zero or negative: an infinity of V times the first is what counts
#pragma unroll
          for (int h = 0; h < G; ++h) o[h] = fabsf(o[h]) == INFINITY ? o[h] : o[h] + o[HB + h];
        bool grew = false;
#pragma unroll
        for (int h = 0; h < G; ++h) grew |= mtile[h] > M[h];
        if (grew)  // the same in every thread
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mn = fmaxf(M[h], mtile[h]);
            acc[h] *= rescale(M[h], mn);
            M[h] = mn;
          }
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float c = rescale(mtile[h], M[h]);
          const float x = tail ? (d < D ? o[h] : 0.f)
                               : fmaf(fmaf(o[2 * HB + h], 0.0625f, o[HB + h]), 0.0625f, o[h]) * 0x1p-8f;
          acc[h] += x * c;
        }
      }
      if (ok && g.ntiles > 0)
        ok = wait.all(bar + B_RFULL + 8 * (ka & 1), (ka >> 1) & 1);
      ok = all_of(3, 128, ok);
      if (!ok) {
        if (!g.whole) {
          if (te == 0) misc[M_VALID + si] = 0;
          asm volatile("bar.arrive %0, 160;" ::"r"(4 + si) : "memory");
          ++si;
        }
        continue;
      }
      float ml[G], L[G];  // the segment's largest logit and normaliser
#pragma unroll
      for (int h = 0; h < G; ++h) ml[h] = -INFINITY, L[h] = 0.f;
      if (g.ntiles > 0) {
        const int rb = ka & 1;
        if (te < 8 * G) {  // eight lanes a head, one softmax warp each
          const float2 x = stat[(rb * 8 + (te & 7)) * 8 + (te >> 3)];
          float m = x.x;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
          float l = x.y * (x.x == -INFINITY ? 1.f : ex2(x.x - m));  // a warp without rows has 0
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(lanes, l, o);
          if ((te & 7) == 0) mlb[te >> 3] = make_float4(m, l, 1.f / l, 0.f);
        }
        named_bar(3, 128);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float4 x = mlb[h];
          ml[h] = x.x, L[h] = x.y;
          // relative to the largest logit, V's scale applied; a whole unit's normalised at once
          acc[h] *= g.whole ? rescale(M[h], ml[h]) * x.z : rescale(M[h], ml[h]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + B_REMPTY + 8 * rb);
        ++ka;
      }
      if (D == 64) {  // the rows' second keys join their first ones
        if (d >= D)
#pragma unroll
          for (int h = 0; h < G; ++h) xh[(d - D) * G + h] = acc[h];
        named_bar(3, 128);
        if (d < D)
#pragma unroll
          for (int h = 0; h < G; ++h) acc[h] += xh[d * G + h];
      }
      if (opaque(g.whole)) {
        if (d < D)
#pragma unroll
          for (int h = 0; h < G; ++h)
            if (h < p.ga)
              p.out[((size_t)g.u * p.ga + h) * D + d] = __float2bfloat16(acc[h]);  // no tiles: 0
      } else {
        // its first result if the unit began before this CTA's slots, else its second
        const int slot = 2 * b + (C > 0 || s0 >= (g.u == u_first ? p_first : p_last) ? 0 : 1);
        if (d < D) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            p.part_o[((size_t)slot * G + h) * D + d] = acc[h];
            if (d == 0) p.part_ml[slot * G + h] = make_float2(ml[h], L[h]);
          }
        }
        if (te == 0) misc[M_VALID + si] = 1;
        asm volatile("bar.arrive %0, 160;" ::"r"(4 + si) : "memory");  // W_M counts it
        ++si;
      }
      if (g.tail && g.add && g.tail_old == KB8 - 1)  // the new row completes a block
        complete<D>(p, g.u, g.n0 / KB8, kept_rows(g.u), reinterpret_cast<uint32_t *>(const_cast<int *>(misc + M_RED)), te);
    }
  } else {
    // ---------------- shared units ----------------
    // The CTA that finishes a shared unit's last segment merges them: this warp, while the
    // others stream on (a fence and a count take microseconds behind the tiles), or the whole
    // CTA at its end.  Only the first two segments of a CTA can be of shared units.
    int si = 0;
    auto count_shared = [&](int k) {
      const Seg g = seg_at(k);
      if (g.whole) return;
      named_bar(4 + si, 160);  // the output warps have written (and arrived)
      if (misc[M_VALID + si]) {
        const Shared x = shared_at(g);
        int old = 0;
        __threadfence();
        if (lane == 0) old = atomicAdd(&p.cnt[g.u], 1);
        old = __shfl_sync(0xffffffffu, old, 0);
        if (old == x.nseg - 1) {
          __threadfence();
          if (lane == 0) p.cnt[g.u] = 0;
          if (x.nseg <= FEW && k < nu - 1) merge_few<D, G>(p.part_ml, p.part_o, p.out, p.ga, x, lane, 32);
          else if (lane == 0)
            misc[M_TODO + 4 * si] = x.u, misc[M_TODO + 4 * si + 1] = x.nseg,
                              misc[M_TODO + 4 * si + 2] = x.first, misc[M_TODO + 4 * si + 3] = x.next;
        }
      }
      ++si;
    };
#pragma unroll 1
    for (int k = 0; k < min(nu, 2); ++k) count_shared(k);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_S) tmem_dealloc(tmem, TMEM_COLS);
#pragma unroll 1
  for (int i = 0; i < 2; ++i)  // the ring is free: its memory serves the merge
    if (misc[M_TODO + 4 * i + 1]) {
      const Shared x{misc[M_TODO + 4 * i], misc[M_TODO + 4 * i + 1], misc[M_TODO + 4 * i + 2], misc[M_TODO + 4 * i + 3]};
      if (x.nseg <= FEW) merge_few<D, G>(p.part_ml, p.part_o, p.out, p.ga, x, tid, NTH);
      else merge_cta<D, G>(p, x, reinterpret_cast<float *>(smem), tid);
    }
}

int padded(int G) { return G <= 1 ? 1 : (G <= 2 ? 2 : (G <= 4 ? 4 : 8)); }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int G>
cudaError_t launch_t(const Ctx &c, const Kv8DecodeArgs &a, const P8 &p) {
  using Gm = Geo<D, G>;
  static bool attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<D, G>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  Maps m;
  const uint64_t rows = (uint64_t)a.c.units * a.c.cap / Gm::KPR, trows = (uint64_t)a.c.units * KB8;
  if (!encode_bytes_map(&m.k, a.c.kq, rows, TROWS) || !encode_bytes_map(&m.v, a.c.vq, rows, TROWS) ||
      !encode_bytes_map(&m.k1, a.c.kq, rows, Gm::BR) || !encode_bytes_map(&m.v1, a.c.vq, rows, Gm::BR) ||
      !encode_rows_map(&m.kt, a.c.kt, trows, D, 16) || !encode_rows_map(&m.vt, a.c.vt, trows, D, 16))
    return cudaErrorInvalidValue;
  m.kl = m.kt, m.vl = m.vt;  // not used without kept rows
  const uint64_t lrows = (uint64_t)a.c.units * KL8;
  if (a.c.blocks && (!encode_rows_map(&m.kl, a.c.kl, lrows, D, 16) || !encode_rows_map(&m.vl, a.c.vl, lrows, D, 16)))
    return cudaErrorInvalidValue;
  const long long slots = (long long)a.c.units * (a.c.cap / KB8 + 1);
  long long grid = c.num_sms < MAXCTA ? c.num_sms : MAXCTA;
  if (grid > slots) grid = slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = Gm::SMEM;
  cfg.stream = c.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D, G>, m, p);
}

}  // namespace

// Scratch: the planning count, the shared units' counts and the row counts' copy (zero, zero
// and anything between calls), then two partial results a CTA.
size_t kv8_decode_ws_bytes(long long units, int G, int D) {
  const size_t g = (size_t)padded(G);
  return 256 + 2 * up256((size_t)units * 4) + up256(2 * MAXCTA * g * sizeof(float2)) +
         2 * MAXCTA * g * (size_t)D * sizeof(float);
}

int *kv8_unit_counts(void *ws) { return reinterpret_cast<int *>(static_cast<uint8_t *>(ws) + 256); }

cudaError_t launch_kv8_decode(const Ctx &c, const Kv8DecodeArgs &a) {
  const int Gp = padded(a.G);
  P8 p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k_new = static_cast<const __nv_bfloat16 *>(a.k_new);
  p.v_new = static_cast<const __nv_bfloat16 *>(a.v_new);
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.c = a.c;
  p.lc = (float)(1.4426950408889634 / sqrt((double)a.c.D));
  p.ga = a.G;
  p.new_pos = a.new_pos;
  uint8_t *w = static_cast<uint8_t *>(a.ws);
  p.planned = reinterpret_cast<int *>(w);
  w += 256;
  p.cnt = reinterpret_cast<int *>(w);
  w += up256((size_t)a.c.units * 4);
  p.snap = reinterpret_cast<int *>(w);
  w += up256((size_t)a.c.units * 4);
  p.part_ml = reinterpret_cast<float2 *>(w);
  w += up256(2 * MAXCTA * (size_t)Gp * sizeof(float2));
  p.part_o = reinterpret_cast<float *>(w);
  p.status = c.status;
  p.timeout = c.timeout_ns;
#define KV8_DEC(DD, GG) \
  if (a.c.D == DD && Gp == GG) return launch_t<DD, GG>(c, a, p);
  KV8_DEC(128, 1) KV8_DEC(128, 2) KV8_DEC(128, 4) KV8_DEC(128, 8)
  KV8_DEC(64, 1) KV8_DEC(64, 2) KV8_DEC(64, 4) KV8_DEC(64, 8)
#undef KV8_DEC
  return cudaErrorInvalidValue;
}

}  // namespace kvc
