// cache_api.cu -- host runtime of the calls around the 8-bit cache: argument
// checks, the choice of kernel and of the division of work, and launches on
// the caller's stream.  Nothing here allocates or synchronises.
#include <math.h>

#include <utility>

#include "attend.cuh"
#include "hwr_indexer.h"
#include "internal.h"

namespace hwr {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

indexer_status device_status(int* sms) {
  const int n = current_device_sms();
  if (n == 0) return INDEXER_ECUDA;
  if (n < 0) return INDEXER_EDEVICE;
  *sms = n;
  return INDEXER_OK;
}

bool act_ok(int32_t act) { return act == INDEXER_ACT_BF16 || act == INDEXER_ACT_FP16; }

indexer_status view_rotation(const indexer_rotation* r, int D, RotView* v) {
  *v = RotView{nullptr, 0, 0, 0};
  if (!r || r->rot_dim == 0) return INDEXER_OK;
  if (r->rot_dim < 0 || r->rot_dim % 16 != 0 || r->rot_dim > D || r->rows < 1 || !r->table ||
      !aligned(r->table, 16) || (r->interleaved != 0 && r->interleaved != 1))
    return INDEXER_EINVAL;
  *v = RotView{r->table, r->rows, r->rot_dim, r->interleaved};
  return INDEXER_OK;
}

indexer_status view_cache(const indexer_cache* c, CacheView* v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !aligned(c->k, 16) || !aligned(c->v, 16) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return INDEXER_EINVAL;
  if (c->D != 64 && c->D != 128) return INDEXER_EUNSUPPORTED;
  if (c->n_pages < 1 || c->heads < 1 || c->page_size < 1 || c->block < 1 || c->page_size % c->block != 0)
    return INDEXER_EINVAL;
  if ((c->block & (c->block - 1)) != 0 || c->block > 128 || c->page_size > (1 << 20) || c->heads > 1024)
    return INDEXER_EUNSUPPORTED;
  if (c->page_stride < 16 || c->token_stride < 16 || c->head_stride < c->D || c->page_stride % 16 != 0 ||
      c->token_stride % 16 != 0 || c->head_stride % 16 != 0)
    return INDEXER_EINVAL;
  // (before any product of them)
  if ((c->page_size > 1 && c->token_stride > int64_t(1) << 36) || (c->heads > 1 && c->head_stride > int64_t(1) << 36))
    return INDEXER_EUNSUPPORTED;
  // No two rows of D codes share bytes: of pages, tokens and heads, in the order of
  // their strides, each steps over all of the ones before.
  struct {
    int64_t n, stride;
  } dim[3] = {{c->n_pages, c->page_stride}, {c->page_size, c->token_stride}, {c->heads, c->head_stride}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (dim[j].stride > dim[j + 1].stride) std::swap(dim[j], dim[j + 1]);
  __int128 span = c->D;
  for (const auto& d : dim) {
    if (d.n == 1) continue;
    if (d.stride < span) return INDEXER_EINVAL;
    span += static_cast<__int128>(d.n - 1) * d.stride;
  }
  const int64_t tok_span = (c->page_size - 1) * c->token_stride;
  const int64_t inner = tok_span + (c->heads - 1) * c->head_stride + c->D;
  if (c->page_stride > (int64_t(1) << 36) / c->n_pages || inner > (int64_t(1) << 36)) return INDEXER_EUNSUPPORTED;
  // the attention holds a token's offset in 32 bits, in units of 16 bytes
  if ((c->n_pages - 1) * c->page_stride + tok_span >= int64_t(1) << 36) return INDEXER_EUNSUPPORTED;
  if (c->n_pages > INT32_MAX) return INDEXER_EUNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < c->block) ++shift;
  *v = CacheView{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, c->page_stride / 16, c->token_stride / 16,
                 c->head_stride / 16, c->page_size, c->block, shift, c->page_size / c->block, c->heads};
  return INDEXER_OK;
}

indexer_status view_seqs(const indexer_sequences* s, bool pointers, SeqView* v) {
  if (!s || s->S < 0 || s->B < 0 || s->table_pages < 0 || s->table_stride < 0) return INDEXER_EINVAL;
  if (s->S > INT32_MAX || s->B > (1 << 20)) return INDEXER_EUNSUPPORTED;
  if (s->B > 1 && s->table_stride < s->table_pages) return INDEXER_EINVAL;
  if (pointers && s->B > 0 && (!s->cu_q || !s->kv_len || (!s->page_table && s->table_pages > 0)))
    return INDEXER_EINVAL;
  *v = SeqView{s->S, s->cu_q, s->kv_len, s->page_table, s->table_stride, s->table_pages, s->B};
  return INDEXER_OK;
}

// How a call of indexer_cache_attend runs.
struct AttendPlan {
  AttendParams p;
  bool f16;
  int D, rows;   // rows of a tile: up to 16, the streaming kernel
  int grid;
  size_t off_jobs, off_ml, off_o, bytes;
};

indexer_status plan_attend(const indexer_cache* c, const indexer_sequences* s, const indexer_attention* a,
                           bool pointers, AttendPlan* pl) {
  AttendParams& p = pl->p;
  p = AttendParams{};
  indexer_status st = view_cache(c, &p.c);
  if (st != INDEXER_OK) return st;
  st = view_seqs(s, pointers, &p.s);
  if (st != INDEXER_OK) return st;
  if (!a || !act_ok(a->act) || a->Hq < 1 || a->Hq % c->heads != 0 || a->sel_width < 0 || a->max_q < 0 ||
      (a->causal != 0 && a->causal != 1) || !isfinite(a->scale))
    return INDEXER_EINVAL;
  p.test_wait = a->kernel == (INDEXER_ATTEND_TILE | INDEXER_ATTEND_TEST_WAIT_TIMEOUT);
  const int32_t kernel = p.test_wait ? INDEXER_ATTEND_TILE : a->kernel;
  if (kernel < INDEXER_ATTEND_AUTO || kernel > INDEXER_ATTEND_TILE) return INDEXER_EINVAL;
  p.Hq = a->Hq;
  p.G = a->Hq / c->heads;
  if (p.G > 128) return INDEXER_EUNSUPPORTED;
  if (s->S > INT32_MAX / a->Hq) return INDEXER_EUNSUPPORTED;
  if (static_cast<int64_t>(s->table_pages) * c->page_size > INT32_MAX - 256) return INDEXER_EUNSUPPORTED;
  p.max_keys = s->table_pages * c->page_size;
  p.causal = a->causal;
  p.sel_width = a->sel_width;
  p.scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634);
  if (!isfinite(p.scale_log2)) return INDEXER_EINVAL;
  pl->f16 = a->act == INDEXER_ACT_FP16;
  pl->D = c->D;
  int sms = 0;
  st = device_status(&sms);
  if (st != INDEXER_OK) return st;
  // rows that share a pass over the keys: of a query with a selection, of a
  // sequence without
  const int64_t most_rows = a->sel_width ? p.G : static_cast<int64_t>(a->max_q ? a->max_q : s->S) * p.G;
  const int64_t most_keys = a->sel_width ? a->sel_width : p.max_keys;
  // Streaming costs about 0.9 us for every 128 keys and head that a CTA goes
  // over, for every 16 rows; tiles 1.7 us (128 rows) whatever the rows, and some
  // 20 us more a launch: 9 x 5 queries of 8 heads over 6K tokens take 35 and 41
  // us, one query of 64 heads over 1M tokens 258 and 115 us.
  const double units = static_cast<double>(a->sel_width ? s->S : s->B) * c->heads * most_keys / 128 / sms;
  const int64_t passes = (most_rows + 15) / 16;
  const bool tile = kernel == INDEXER_ATTEND_TILE ||
                    (kernel == INDEXER_ATTEND_AUTO && passes > 2 && units * (0.9 * passes - 1.7) > 30);
  const int R = pl->rows = tile ? (most_rows <= 128 ? 128 : 256) : (most_rows <= 8 ? 8 : 16);
  p.sel_tiles = (p.G + R - 1) / R;
  const int64_t tiles = a->sel_width ? s->S * p.sel_tiles : s->S * p.G / R + s->B;
  const int64_t items = tiles * c->heads;
  if (items > INT32_MAX - 1024) return INDEXER_EUNSUPPORTED;
  p.n_tiles = static_cast<int32_t>(tiles);
  const bool stream = R <= 16;
  const int slots = stream ? sms * attend_stream_ctas_per_sm(R) : sms;
  // Fewer (tile, head)s than fill the SMs a few times over: the CTAs share all
  // keys equally, across tiles, and a second kernel joins the parts.
  const bool split = tiles <= (stream ? kMaxSplitTiles : kMaxSplitTiles2) && items < 8 * slots &&
                     tiles * (most_keys / 64 + 1) <= INT32_MAX;
  p.n_ctas = split ? slots : 0;
  // Heads side by side: 16 x 16K..64K tokens of 8 heads 216 us, 258 us head by head.
  p.lanes = split && stream && slots % c->heads * 10 <= slots && slots >= c->heads ? c->heads : 1;
  pl->grid = split ? slots : static_cast<int>(items);
  size_t at = 0;
  pl->off_jobs = at;
  at += split ? align256(static_cast<size_t>(slots) * sizeof(JoinJob)) : 0;
  pl->off_ml = at;
  at += split ? align256(static_cast<size_t>(2) * slots * R * sizeof(float2)) : 0;
  pl->off_o = at;
  at += split ? align256(static_cast<size_t>(2) * slots * R * c->D * sizeof(float)) : 0;
  pl->bytes = at > 256 ? at : 256;
  return INDEXER_OK;
}

}  // namespace
}  // namespace hwr

using namespace hwr;

extern "C" {

indexer_status indexer_rotate_quantise(const void* x, int64_t S, int32_t H, int32_t D, int32_t act, int64_t x_stride,
                                       const int32_t* positions, const indexer_rotation* rotation, uint8_t* codes,
                                       float* scale, int32_t* status, void* stream) {
  if (S < 0 || H < 0 || !act_ok(act)) return INDEXER_EINVAL;
  if (D != 64 && D != 128) return INDEXER_EUNSUPPORTED;
  if (S > INT32_MAX || H > 65535 * 4) return INDEXER_EUNSUPPORTED;
  RotView r;
  indexer_status st = view_rotation(rotation, D, &r);
  if (st != INDEXER_OK) return st;
  if (S == 0 || H == 0) return INDEXER_OK;
  if (!x || !codes || !scale || !aligned(x, 16) || !aligned(codes, 8) || !aligned(scale, 4) || x_stride % 8 != 0 ||
      x_stride < static_cast<int64_t>(H) * D)
    return INDEXER_EINVAL;
  int sms = 0;
  st = device_status(&sms);
  if (st != INDEXER_OK) return st;
  if (launch_rotate_quantise(x, S, H, D, act == INDEXER_ACT_FP16, x_stride, positions, r, codes, scale,
                             reinterpret_cast<uint32_t*>(status), sms, static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return INDEXER_ECUDA;
  return INDEXER_OK;
}

indexer_status indexer_cache_append(const indexer_cache* cache, const indexer_sequences* seqs, const void* k,
                                    const void* v, int64_t kv_stride, int32_t act, const indexer_rotation* rotation,
                                    const void* q, int32_t Hq, int64_t q_stride, void* q_out, int32_t* status,
                                    void* stream) {
  AppendParams p = {};
  indexer_status st = view_cache(cache, &p.c);
  if (st != INDEXER_OK) return st;
  st = view_seqs(seqs, true, &p.s);
  if (st != INDEXER_OK) return st;
  st = view_rotation(rotation, cache->D, &p.r);
  if (st != INDEXER_OK) return st;
  if (!act_ok(act) || (q == nullptr) != (q_out == nullptr)) return INDEXER_EINVAL;
  if (seqs->S > INT32_MAX / cache->heads / cache->D) return INDEXER_EUNSUPPORTED;
  if (seqs->S == 0 || seqs->B == 0) return INDEXER_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || kv_stride % 8 != 0 ||
      kv_stride < static_cast<int64_t>(cache->heads) * cache->D)
    return INDEXER_EINVAL;
  if (q) {
    if (Hq < 1 || !aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 != 0 ||
        q_stride < static_cast<int64_t>(Hq) * cache->D)
      return INDEXER_EINVAL;
    if (seqs->S > INT32_MAX / Hq) return INDEXER_EUNSUPPORTED;
  }
  int sms = 0;
  st = device_status(&sms);
  if (st != INDEXER_OK) return st;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.kv_stride = kv_stride * 2;
  p.q = static_cast<const uint8_t*>(q);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.q_stride = q_stride * 2;
  p.Hq = q ? Hq : 0;
  p.status = reinterpret_cast<uint32_t*>(status);
  if (launch_cache_append(p, cache->D, act == INDEXER_ACT_FP16, sms, static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return INDEXER_ECUDA;
  return INDEXER_OK;
}

indexer_status indexer_cache_attend_workspace_bytes(const indexer_cache* cache, const indexer_sequences* seqs,
                                                    const indexer_attention* attention, size_t* bytes) {
  AttendPlan pl;
  const indexer_status st = plan_attend(cache, seqs, attention, false, &pl);
  if (st != INDEXER_OK) return st;
  if (!bytes) return INDEXER_EINVAL;
  *bytes = pl.bytes;
  return INDEXER_OK;
}

indexer_status indexer_cache_attend(const indexer_cache* cache, const indexer_sequences* seqs,
                                    const indexer_attention* attention, const void* q, int64_t q_stride,
                                    const int32_t* sel_idx, const int32_t* sel_len, void* out, float* lse,
                                    int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  AttendPlan pl;
  const indexer_status st = plan_attend(cache, seqs, attention, true, &pl);
  if (st != INDEXER_OK) return st;
  if (seqs->S == 0 || seqs->B == 0) return INDEXER_OK;
  AttendParams& p = pl.p;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || q_stride % 8 != 0 ||
      q_stride < static_cast<int64_t>(attention->Hq) * cache->D)
    return INDEXER_EINVAL;
  if (attention->sel_width && (!sel_idx || !sel_len)) return INDEXER_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < pl.bytes) return INDEXER_EWORKSPACE;
  p.q = static_cast<const uint8_t*>(q);
  p.q_stride = q_stride * 2;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.sel_idx = sel_idx;
  p.sel_len = sel_len;
  p.status = reinterpret_cast<uint32_t*>(status);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.jobs = reinterpret_cast<JoinJob*>(ws + pl.off_jobs);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + pl.off_o);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool u16 = !p.sel_width && p.c.block % 16 == 0;
  const cudaError_t e = pl.rows <= 16 ? launch_attend_stream(p, pl.D, pl.rows, pl.f16, pl.grid, cs)
                                      : launch_attend_tile(p, pl.D, pl.rows, u16, pl.f16, pl.grid, cs);
  if (e != cudaSuccess) return INDEXER_ECUDA;
  if (p.n_ctas && launch_attend_join(p, pl.D, pl.rows, pl.f16, cs) != cudaSuccess) return INDEXER_ECUDA;
  return INDEXER_OK;
}

}  // extern "C"
