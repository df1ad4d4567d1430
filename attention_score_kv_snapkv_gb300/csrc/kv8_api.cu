// C ABI of the 8-bit KV cache (declared and documented in include/kvcompress.h): host-side
// argument checks, which need no device, then the launches.
#include "kv8.cuh"

namespace kvc {
namespace {

inline bool al(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline kvc_status launched(cudaError_t e) { return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA; }
const long long kMaxRows = (1ll << 31) - 1;
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b && x < y + nb && y < x + na;
}

// Checks the cache's sizes and buffers and fills *c.
kvc_status check_cache(const kvc_kv8_params *p, const kvc_kv8_cache *x, Kv8 *c) {
  if (!p || !x) return KVC_ERR_NULL;
  if (p->n_layers < 1 || p->batch < 1 || p->n_kv_heads < 1 ||
      (p->head_dim != 64 && p->head_dim != 128) || p->cap < 1 || p->cap % KB8)
    return KVC_ERR_SHAPE;
  // each factor is below 2^31, so the product is checked step by step
  long long units = (long long)p->n_layers * p->batch;
  if (units > kMaxRows) return KVC_ERR_SHAPE;
  units *= p->n_kv_heads;
  if (units > kMaxRows || units * p->cap > kMaxRows) return KVC_ERR_SHAPE;
  if (!x->k_codes || !x->v_codes || !x->k_scale || !x->v_scale || !x->k_tail || !x->v_tail || !x->n_valid)
    return KVC_ERR_NULL;
  if (!al(x->k_codes, 16) || !al(x->v_codes, 16) || !al(x->k_tail, 16) || !al(x->v_tail, 16) ||
      !al(x->k_scale, 4) || !al(x->v_scale, 4) || !al(x->n_valid, 4) || !al(x->pos, 4) ||
      !al(x->k_last, 16) || !al(x->v_last, 16) || !al(x->blocks, 8))
    return KVC_ERR_ALIGN;
  if (!x->k_last != !x->blocks || !x->v_last != !x->blocks) return KVC_ERR_NULL;  // all or none
  c->kq = static_cast<uint8_t *>(x->k_codes);
  c->vq = static_cast<uint8_t *>(x->v_codes);
  c->ks = x->k_scale;
  c->vs = x->v_scale;
  c->kt = static_cast<__nv_bfloat16 *>(x->k_tail);
  c->vt = static_cast<__nv_bfloat16 *>(x->v_tail);
  c->pos = x->pos;
  c->n_valid = x->n_valid;
  c->kl = static_cast<__nv_bfloat16 *>(x->k_last);
  c->vl = static_cast<__nv_bfloat16 *>(x->v_last);
  c->blocks = reinterpret_cast<int2 *>(x->blocks);
  c->units = (int)units;
  c->D = p->head_dim;
  c->cap = p->cap;
  return KVC_OK;
}

// The scratch of a step for G query heads a KV head (its counts for any).
kvc_status check_scratch(const kvc_kv8_params *p, const kvc_kv8_cache *x, int G) {
  const long long units = (long long)p->n_layers * p->batch * p->n_kv_heads;
  if (units > KVC_DECODE_MAX_UNITS) return KVC_ERR_SHAPE;
  if (!x->scratch || x->scratch_bytes < kv8_decode_ws_bytes(units, G, p->head_dim)) return KVC_ERR_WORKSPACE;
  return al(x->scratch, 256) ? KVC_OK : KVC_ERR_ALIGN;
}

// SnapKV's selection into the cache: votes formed from q_win, or given.
kvc_status snapkv_kv8(const kvc_snapkv_params *p, const void *q_win, const float *votes, const void *k,
                      const void *v, const kvc_kv8_cache *cache, float *votes_out, void *workspace,
                      size_t workspace_bytes, kvc_stream_t stream) {
  if (!p) return KVC_ERR_NULL;
  const kvc_kv8_params kp = {p->n_layers, p->batch, p->n_q_heads, p->n_kv_heads, p->head_dim, p->cap, 0};
  Kv8WriteArgs a;
  kvc_status st = check_cache(&kp, cache, &a.c);
  if (st != KVC_OK) return st;
  if (!k || !v || !a.c.pos) return KVC_ERR_NULL;
  const void *v_dev = nullptr;
  st = snapkv_positions(p, q_win, votes, k, v, a.c.pos, a.c.n_valid, votes_out, workspace,
                        workspace_bytes, stream, &v_dev);
  if (st != KVC_OK) return st;
  Ctx c;
  st = make_ctx(stream, &c);
  if (st != KVC_OK) return st;
  const bool all = p->budget >= p->prompt_len || p->keep_window >= p->prompt_len;
  a.k = k;
  a.v = v_dev;
  a.rows = a.c.pos;
  a.rows_ld = p->cap;
  a.pos_in = nullptr;
  a.lengths = nullptr;
  a.L = p->prompt_len;
  a.n_rows = all ? p->prompt_len : p->budget;
  a.set_state = 0;  // the selection wrote the positions and the row counts
  return launched(launch_kv8_write(c, a));
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

size_t kv8_scratch_bytes(const kvc_kv8_params *p) {
  if (!p || p->n_layers < 1 || p->batch < 1 || p->n_kv_heads < 1 || p->n_q_heads < 1 ||
      p->n_q_heads % p->n_kv_heads || (p->head_dim != 64 && p->head_dim != 128))
    return 256;
  const long long units = (long long)p->n_layers * p->batch * p->n_kv_heads;
  if ((long long)p->n_layers * p->batch > KVC_DECODE_MAX_UNITS || units > KVC_DECODE_MAX_UNITS) return 256;
  return kv8_decode_ws_bytes(units, p->n_q_heads / p->n_kv_heads, p->head_dim);
}

kvc_status kv8_write(const kvc_kv8_params *p, int32_t src_len, int32_t n_rows, const void *k,
                     const void *v, const int32_t *rows, const int32_t *pos, const int32_t *lengths,
                     const kvc_kv8_cache *cache, kvc_stream_t stream) {
  const TraceRange trace_range("kv8_write");
  Kv8WriteArgs a;
  kvc_status st = check_cache(p, cache, &a.c);
  if (st != KVC_OK) return st;
  if (src_len < 1 || n_rows < 1 || (!rows && n_rows > src_len) || (long long)a.c.units * src_len > kMaxRows)
    return KVC_ERR_SHAPE;
  if (n_rows > p->cap) return KVC_ERR_BUDGET;
  if (!k || !v || (pos && !a.c.pos)) return KVC_ERR_NULL;
  if (!al(k, 16) || !al(v, 16) || !al(rows, 4) || !al(pos, 4) || !al(lengths, 4)) return KVC_ERR_ALIGN;
  Ctx c;
  st = make_ctx(stream, &c);
  if (st != KVC_OK) return st;
  a.k = k;
  a.v = v;
  a.rows = rows;
  a.rows_ld = n_rows;
  a.pos_in = pos;
  a.lengths = lengths;
  a.L = src_len;
  a.n_rows = n_rows;
  a.set_state = 1;
  return launched(launch_kv8_write(c, a));
}

kvc_status kv8_append(const kvc_kv8_params *p, int32_t m, const void *k_new, const void *v_new,
                      const int32_t *counts, const kvc_kv8_cache *cache, kvc_stream_t stream) {
  const TraceRange trace_range("kv8_append");
  Kv8AppendArgs a;
  kvc_status st = check_cache(p, cache, &a.c);
  if (st != KVC_OK) return st;
  if (m < 1 || p->new_pos < 0 || (long long)a.c.units * m > kMaxRows || (long long)p->new_pos + m > kMaxRows)
    return KVC_ERR_SHAPE;
  if (!k_new || !v_new) return KVC_ERR_NULL;
  if (!al(k_new, 16) || !al(v_new, 16) || !al(counts, 4)) return KVC_ERR_ALIGN;
  st = check_scratch(p, cache, 1);
  if (st != KVC_OK) return st;
  Ctx c;
  st = make_ctx(stream, &c);
  if (st != KVC_OK) return st;
  a.k = k_new;
  a.v = v_new;
  a.counts = counts;
  a.m = m;
  a.new_pos = p->new_pos;
  a.cnt = kv8_unit_counts(cache->scratch);
  return launched(launch_kv8_append(c, a));
}

kvc_status kv8_read(const kvc_kv8_params *p, const kvc_kv8_cache *cache, int32_t out_rows, void *k_out,
                    void *v_out, kvc_stream_t stream) {
  const TraceRange trace_range("kv8_read");
  Kv8ReadArgs a;
  kvc_status st = check_cache(p, cache, &a.c);
  if (st != KVC_OK) return st;
  if (out_rows < 1 || (long long)a.c.units * out_rows > kMaxRows) return KVC_ERR_SHAPE;
  if (!k_out || !v_out) return KVC_ERR_NULL;
  if (!al(k_out, 16) || !al(v_out, 16)) return KVC_ERR_ALIGN;
  Ctx c;
  st = make_ctx(stream, &c);
  if (st != KVC_OK) return st;
  a.k = k_out;
  a.v = v_out;
  a.out_rows = out_rows;
  return launched(launch_kv8_read(c, a));
}

kvc_status kv8_decode_attn(const kvc_kv8_params *p, const void *q, const void *k_new, const void *v_new,
                           const kvc_kv8_cache *cache, void *out, kvc_stream_t stream) {
  const TraceRange trace_range("kv8_decode_attn");
  Kv8DecodeArgs a;
  kvc_status st = check_cache(p, cache, &a.c);
  if (st != KVC_OK) return st;
  if (p->n_q_heads < 1 || p->n_q_heads % p->n_kv_heads || p->n_q_heads / p->n_kv_heads > 8 ||
      a.c.units > KVC_DECODE_MAX_UNITS || p->new_pos < 0)
    return KVC_ERR_SHAPE;
  if (!q || !out || (k_new == nullptr) != (v_new == nullptr)) return KVC_ERR_NULL;
  if (!al(q, 16) || !al(out, 16) || !al(k_new, 16) || !al(v_new, 16)) return KVC_ERR_ALIGN;
  // a unit's queries are read before its output is written, but other units' rows are not
  const size_t row = (size_t)p->head_dim * 2, nk = a.c.units * row, nq = nk * (p->n_q_heads / p->n_kv_heads);
  if ((out != q && overlap(out, nq, q, nq)) || overlap(out, nq, k_new, nk) || overlap(out, nq, v_new, nk))
    return KVC_ERR_SHAPE;
  st = check_scratch(p, cache, p->n_q_heads / p->n_kv_heads);
  if (st != KVC_OK) return st;
  Ctx c;
  st = make_ctx(stream, &c);
  if (st != KVC_OK) return st;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.out = out;
  a.ws = cache->scratch;
  a.G = p->n_q_heads / p->n_kv_heads;
  a.new_pos = p->new_pos;
  return launched(launch_kv8_decode(c, a));
}

kvc_status snapkv_select_kv8(const kvc_snapkv_params *p, const float *votes, const void *k, const void *v,
                             const kvc_kv8_cache *cache, void *workspace, size_t workspace_bytes,
                             kvc_stream_t stream) {
  const TraceRange trace_range("snapkv_select_kv8");
  if (!votes) return KVC_ERR_NULL;
  return snapkv_kv8(p, nullptr, votes, k, v, cache, nullptr, workspace, workspace_bytes, stream);
}

kvc_status snapkv_compress_kv8(const kvc_snapkv_params *p, const void *q_win, const void *k, const void *v,
                               const kvc_kv8_cache *cache, float *votes_out, void *workspace,
                               size_t workspace_bytes, kvc_stream_t stream) {
  const TraceRange trace_range("snapkv_compress_kv8");
  if (!q_win) return KVC_ERR_NULL;
  return snapkv_kv8(p, q_win, nullptr, k, v, cache, votes_out, workspace, workspace_bytes, stream);
}

}  // extern "C"
