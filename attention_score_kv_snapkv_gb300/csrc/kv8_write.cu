// Writing and reading the 8-bit KV cache: bf16 rows to e4m3 codes with one power-of-two
// scale for each block of KVC_KV8_BLOCK rows of a unit (K and V apart), and back.  The rows
// past the last whole block stay in bf16 in the unit's tail until later rows fill the block,
// so what the cache holds depends on the rows alone, not on how many calls brought them,
// and no row is rounded twice.
//
// All three are bound by HBM: 6 bytes an element (2 read, 1 written for K and for V, or the
// reverse).  One CTA of 128 threads takes one block of K or V (of 64-wide rows both): its rows
// (16 KB) are held in registers, eight 16-byte loads a thread in flight, so a block is read
// once for both its largest magnitude and its codes.
#include "kv8.cuh"

namespace kvc {
namespace {

// The write and the append may be launched while the kernel before them in the stream still runs,
// and wait for it (an append of 700 rows 8.7 us against 9.4).  They let the next one be launched
// only by ending: an early trigger made a selection every time 38.7 us instead of 34.7; and the
// read-back, one short wave, took 3.8 us so and 2.8 launched plainly.  Their sources may have been
// written by the kernel that they overlap, so they are not loaded by way of the read-only cache, whose
// lines that kernel's end does not renew.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_overlapped(cudaStream_t stream, unsigned grid, void (*kernel)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(KV8_NT);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The kept copy of the tail's first row, and the rows of the block completed last before it.
__device__ __forceinline__ uint4 *last_rows(const Kv8 &c, int u, bool is_v) {
  return reinterpret_cast<uint4 *>(is_v ? c.vl : c.kl) + (size_t)u * KL8 * (c.D / 8);
}
__device__ __forceinline__ uint4 *first_row(const Kv8 &c, int u, bool is_v) {
  return last_rows(c, u, is_v) + KB8 * (c.D / 8);
}

// Grid: units x blocks x {K, V}, K and V of a block next to each other; a CTA takes both where
// rows are 64 wide (half as much each: as many bytes in flight, half as many CTAs).  Loads are
// without branches, so that all of a thread's are in flight at once.
// Measured (GB300, graph of calls on three sources in turn): 128 units of 16384 rows, D = 128,
// 225 us (1.61 GB, 7.2 TB/s: 107% of the measured copy), D = 64 115 us; 192 ragged units of up to
// 1023 rows, D = 64, 8.1 us (71%).  One load behind each branch took 285 us for the first (a
// persistent CTA an SM with a ring of bulk copies 261) and 153 us for the second.
// 10 CTAs an SM (48 registers, no spills): with 12 (40 registers) 52 to 104 bytes spill, 229 and 117
// us; with 8 a selection of 1024 of 16384 rows takes 36.4 us, with 10 34.5.
template <int D>
__global__ void __launch_bounds__(KV8_NT, 10) kv8_write_kernel(const Kv8WriteArgs a, uint32_t *status) {
  constexpr int RV = D / 8, NP = KB8 * RV / KV8_NT, RS = KV8_NT / RV;  // RS rows a step
  constexpr int NX = 128 / D;                                          // K and V: 1 or both
  wait_for_stream();
  const int t = threadIdx.x;
  const int nb = (a.n_rows + KB8 - 1) / KB8;
  const int first = NX == 1 ? blockIdx.x & 1 : 0, item = NX == 1 ? blockIdx.x >> 1 : blockIdx.x;  // first: 0 K, 1 V
  const int u = item / nb, b = item - u * nb;
  int n = a.n_rows;
  if (a.lengths) {
    n = a.lengths[u];
    if (n < 0 || n > a.n_rows) {
      if (t == 0 && b == 0) set_status(status, KVC_DEV_BAD_STATE);
      n = n < 0 ? 0 : a.n_rows;
    }
  }
  const int32_t *map = a.rows ? a.rows + (size_t)u * a.rows_ld : nullptr;
  if (a.set_state && first == 0) {
    const int end = b == nb - 1 ? a.c.cap : (b + 1) * KB8;  // the last one clears what is behind
    if (a.c.pos)
      for (int r = b * KB8 + t; r < end; r += KV8_NT)
        a.c.pos[(size_t)u * a.c.cap + r] =
            r >= n ? -1 : (a.pos_in ? a.pos_in[(size_t)u * a.n_rows + r] : (map ? map[r] : r));
    if (b == 0 && t == 0) a.c.n_valid[u] = n;
  }
  if (a.c.blocks && first == 0 && b == 0 && t == 0) a.c.blocks[u] = make_int2(n / KB8, -1);
  if (b * KB8 >= n) return;
  const int piece = t % RV, row0 = t / RV;
  uint4 w[NX][NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = b * KB8 + row0 + i * RS;
    const int s = r < n ? (map ? map[r] : r) : -1;
    const bool in = s >= 0 && s < a.L;
    if (r < n && !in && piece == 0) set_status(status, KVC_DEV_BAD_STATE);  // outside the source: zeros
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const uint4 *src = reinterpret_cast<const uint4 *>(first + x ? a.v : a.k) + (size_t)u * a.L * RV;
      w[x][i] = in ? __ldcg(src + (size_t)s * RV + piece) : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int x = 0; x < NX; ++x) {
    const bool is_v = first + x;
    if ((b + 1) * KB8 <= n) {
      __shared__ uint32_t red[4];
      uint8_t *dst = (is_v ? a.c.vq : a.c.kq) + ((size_t)u * a.c.cap + (size_t)b * KB8) * D;
      float *sc = (is_v ? a.c.vs : a.c.ks) + (size_t)u * (a.c.cap / KB8) + b;
      quantise_block<D>(w[x], dst, sc, red, 1, t);
      if (a.c.blocks && (b + 1) * KB8 == n && t < RV)  // no open rows: the tail stays as it was
        first_row(a.c, u, is_v)[t] = __ldcg(reinterpret_cast<const uint4 *>(is_v ? a.c.vt : a.c.kt) +
                                            (size_t)u * KB8 * RV + t);
    } else {
      uint4 *tail = reinterpret_cast<uint4 *>(is_v ? a.c.vt : a.c.kt) + (size_t)u * KB8 * RV;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (b * KB8 + row0 + i * RS < n) tail[t + i * KV8_NT] = w[x][i];
      if (a.c.blocks && t < RV) first_row(a.c, u, is_v)[t] = w[x][0];
    }
  }
}

// Adds rows to every unit.  Grid: units x {K, V} x CTAs; CTA j takes the j-th block that fills,
// and CTA 0, whose block starts with the tail's rows, then writes the new tail.  The row count
// changes when every CTA of the unit has read it: the last one to count itself writes it.
// The rows of one completed block are kept as they came, so that the row count may be lowered into
// it: the block that held rows before, else the last one (64 units of 700 rows: 32 KB
// a unit more to 537; 8.9 us, without them and the first row's copy 7.3).
template <int D>
__global__ void __launch_bounds__(KV8_NT) kv8_append_kernel(const Kv8AppendArgs a, int per, uint32_t *status) {
  constexpr int RV = D / 8, NP = KB8 * RV / KV8_NT, RS = KV8_NT / RV;
  __shared__ uint32_t red[4];
  const int t = threadIdx.x, u = blockIdx.x / (2 * per), x = blockIdx.x - u * 2 * per, j = x >> 1;
  const bool is_v = x & 1;
  wait_for_stream();
  const int piece = t % RV, row0 = t / RV;
  uint4 *tail = reinterpret_cast<uint4 *>(is_v ? a.c.vt : a.c.kt) + (size_t)u * KB8 * RV;
  uint4 head = make_uint4(0, 0, 0, 0), copy = head;  // the tail's first row, and its copy
  if (a.c.blocks && j == 0 && t < RV) head = tail[t], copy = first_row(a.c, u, is_v)[t];
  const int2 blk = a.c.blocks ? a.c.blocks[u] : make_int2(-1, -1);
  int n0 = a.c.n_valid[u];
  int m = a.counts ? a.counts[u] : a.m;
  bool bad = false, full = false;
  if (n0 < 0 || n0 > a.c.cap) bad = true, n0 = n0 < 0 ? 0 : a.c.cap;
  if (m < 0 || m > a.m) bad = true, m = m < 0 ? 0 : a.m;
  if (m > a.c.cap - n0) full = true, m = a.c.cap - n0;
  if (x == 0 && t == 0 && (bad || full))
    set_status(status, (bad ? KVC_DEV_BAD_STATE : 0u) | (full ? KVC_DEV_CACHE_FULL : 0u));
  const int n1 = n0 + m, b = n0 / KB8 + j, last = n1 / KB8;
  const uint4 *src = reinterpret_cast<const uint4 *>(is_v ? a.v : a.k) + (size_t)u * a.m * RV;
  const bool fills = b < last;
  const int keep = n0 % KB8 ? n0 / KB8 : last - 1;        // the completed block whose rows are kept
  const bool opens = a.c.blocks && j == 0 && m > 0;       // this CTA leaves the tail's first row
  const int open = opens ? open_rows(n0, blk) : OPEN_TAIL;
  uint4 w[NP];
  const uint4 *old = tail;                                // the open block's rows
  if (open != OPEN_TAIL && __syncthreads_and(same16(head, copy))) {
    if (open == OPEN_LAST) old = last_rows(a.c, u, is_v);
    else if (t == 0) set_status(status, KVC_DEV_BAD_STATE);
  }
  if (fills) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = b * KB8 + row0 + i * RS;
      w[i] = r < n0 ? old[t + i * KV8_NT] : __ldcg(src + (size_t)(r - n0) * RV + piece);
    }
  }
  __syncthreads();  // every thread has read the row count, and the tail if it is to be read
  if (t == 0) {
    __threadfence();
    if (atomicAdd(a.cnt + u, 1) == 2 * per - 1) {
      a.cnt[u] = 0;
      a.c.n_valid[u] = n1;
      if (a.c.blocks && m > 0)
        a.c.blocks[u] = make_int2(last, last > n0 / KB8 ? keep : (blk.x == n0 / KB8 ? blk.y : -1));
    }
  }
  if (fills) {
    if (a.c.blocks && b == keep) {
#pragma unroll
      for (int i = 0; i < NP; ++i) last_rows(a.c, u, is_v)[t + i * KV8_NT] = w[i];
    }
    uint8_t *dst = (is_v ? a.c.vq : a.c.kq) + ((size_t)u * a.c.cap + (size_t)b * KB8) * D;
    quantise_block<D>(w, dst, (is_v ? a.c.vs : a.c.ks) + (size_t)u * (a.c.cap / KB8) + b, red, 1, t);
  }
  if (j == 0) {  // the open block's new rows; rows of the tail behind them stay as they were
    const int from = old != tail && !fills ? last * KB8 : n0;  // rows that are not in the tail yet
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = last * KB8 + row0 + i * RS;
      w[i] = r >= n0 && r < n1 ? __ldcg(src + (size_t)(r - n0) * RV + piece)
                               : (r >= from && r < n0 ? old[t + i * KV8_NT] : make_uint4(0, 0, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = last * KB8 + row0 + i * RS;
      if (r >= from && r < n1) tail[t + i * KV8_NT] = w[i];
    }
    if (opens && t < RV) first_row(a.c, u, is_v)[t] = last * KB8 >= from && last * KB8 < n1 ? w[0] : head;
  }
  if (!is_v && a.c.pos)
    for (int r = n0 + j * KV8_NT + t; r < n1; r += per * KV8_NT)
      a.c.pos[(size_t)u * a.c.cap + r] = a.new_pos + (r - n0);
}

template <int D>
__global__ void __launch_bounds__(KV8_NT) kv8_read_kernel(const Kv8ReadArgs a, int nb, uint32_t *status) {
  constexpr int RV = D / 8, NP = KB8 * RV / KV8_NT, RS = KV8_NT / RV;
  const int t = threadIdx.x;
  const bool is_v = blockIdx.x & 1;
  const int u = (blockIdx.x >> 1) / nb, b = (blockIdx.x >> 1) - u * nb;
  int n = a.c.n_valid[u];
  if (n < 0 || n > a.c.cap) {
    if (t == 0 && b == 0) set_status(status, KVC_DEV_BAD_STATE);
    n = n < 0 ? 0 : a.c.cap;
  }
  const int whole = n / KB8;
  const int lim = min(n, a.out_rows);
  if (b * KB8 >= lim) return;
  const uint4 *tail = reinterpret_cast<const uint4 *>(is_v ? a.c.vt : a.c.kt) + (size_t)u * KB8 * RV;
  if (b == whole && a.c.blocks) {
    const int open = open_rows(n, a.c.blocks[u]);
    if (open != OPEN_TAIL && __syncthreads_and(t >= RV || same16(tail[t], first_row(a.c, u, is_v)[t]))) {
      if (open == OPEN_LAST) tail = last_rows(a.c, u, is_v);
      else if (t == 0) set_status(status, KVC_DEV_BAD_STATE);
    }
  }
  const int row0 = t / RV;
  uint4 *dst = reinterpret_cast<uint4 *>(is_v ? a.v : a.k) + ((size_t)u * a.out_rows + (size_t)b * KB8) * RV;
  if (b < whole) {
    const uint2 *src = reinterpret_cast<const uint2 *>(is_v ? a.c.vq : a.c.kq) +
                       ((size_t)u * a.c.cap + (size_t)b * KB8) * RV;
    uint2 w[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) w[i] = __ldg(src + t + i * KV8_NT);
    const float s = __ldg((is_v ? a.c.vs : a.c.ks) + (size_t)u * (a.c.cap / KB8) + b);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      uint4 o;
      uint32_t *op = &o.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_float(((j < 2 ? w[i].x : w[i].y) >> ((j & 1) * 16)) & 0xffffu);
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact: 4 significant bits
        op[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
      if (b * KB8 + row0 + i * RS < lim) dst[t + i * KV8_NT] = o;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (b * KB8 + row0 + i * RS < lim) dst[t + i * KV8_NT] = tail[t + i * KV8_NT];
  }
}

}  // namespace

cudaError_t launch_kv8_write(const Ctx &c, const Kv8WriteArgs &a) {
  const long long blocks = 2ll * a.c.units * ((a.n_rows + KB8 - 1) / KB8);
  return a.c.D == 128 ? launch_overlapped(c.stream, (unsigned)blocks, kv8_write_kernel<128>, a, c.status)
                      : launch_overlapped(c.stream, (unsigned)(blocks / 2), kv8_write_kernel<64>, a, c.status);
}

cudaError_t launch_kv8_append(const Ctx &c, const Kv8AppendArgs &a) {
  const int per = a.m < KB8 ? 1 : (KB8 - 1 + a.m) / KB8;  // blocks that m rows can fill
  const unsigned grid = (unsigned)(2ll * a.c.units * per);
  return a.c.D == 128 ? launch_overlapped(c.stream, grid, kv8_append_kernel<128>, a, per, c.status)
                      : launch_overlapped(c.stream, grid, kv8_append_kernel<64>, a, per, c.status);
}

cudaError_t launch_kv8_read(const Ctx &c, const Kv8ReadArgs &a) {
  const int rows = a.out_rows < a.c.cap ? a.out_rows : a.c.cap;
  const int nb = (rows + KB8 - 1) / KB8;
  const unsigned grid = (unsigned)(2ll * a.c.units * nb);
  if (a.c.D == 128)
    kv8_read_kernel<128><<<grid, KV8_NT, 0, c.stream>>>(a, nb, c.status);
  else
    kv8_read_kernel<64><<<grid, KV8_NT, 0, c.stream>>>(a, nb, c.status);
  return cudaGetLastError();
}

}  // namespace kvc
