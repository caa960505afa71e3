// kv_api.cu -- the extern "C" boundary of include/fakv.h: argument checks and dispatch.
#include <cmath>
#include <initializer_list>
#include "kv_quant.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int MAX_SEQS = 16384;
constexpr double MAX_BYTES = 1125899906842624.0;  // 2^50, as in fa.h

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool dtype_ok(fa_dtype t) { return t == FA_F32 || t == FA_BF16; }

// Any stride below 2^50 bytes and not negative: no offset computed from it can wrap.
bool stride_ok(long long s, int es) { return s >= 0 && (double)s * es <= MAX_BYTES; }

fa_status check_cache(const fakv_cache* c) {
  if (!c || !dtype_ok(c->dtype)) return FA_ERR_INVALID_ARG;
  if (c->planes < 1 || c->num_pages < 1 || c->HKV < 1 || c->D < 1 || c->max_slots < 1 || c->max_pages < 1 ||
      c->page_size < 1)
    return FA_ERR_INVALID_ARG;
  if (c->D % 16 != 0 || c->D > 128) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return FA_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > (1ll << 30) || c->num_pages > (1 << 28) || c->HKV > 65535 ||
      c->max_slots > (1 << 28))
    return FA_ERR_INVALID_ARG;
  const int es = esize(c->dtype);
  for (long long s : {c->page_stride, c->token_stride, c->head_stride}) {
    if (s <= 0 || !stride_ok(s, es)) return FA_ERR_INVALID_ARG;
    if (s * es % 16 != 0) return FA_ERR_ALIGNMENT;
  }
  if (c->planes > 1) {
    if (c->plane_stride <= 0 || !stride_ok(c->plane_stride, es)) return FA_ERR_INVALID_ARG;
    if (c->plane_stride * es % 16 != 0) return FA_ERR_ALIGNMENT;
    if ((double)c->planes * c->plane_stride * es > MAX_BYTES) return FA_ERR_INVALID_ARG;
  }
  if ((double)c->num_pages * c->page_stride * es > MAX_BYTES) return FA_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages || (double)c->max_slots * c->table_stride * 4 > MAX_BYTES)
    return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)c->K, (const void*)c->V, (const void*)c->table, (const void*)c->lens}) {
    if (!p) return FA_ERR_INVALID_ARG;
  }
  if (!aligned(c->K, 16) || !aligned(c->V, 16)) return FA_ERR_ALIGNMENT;
  if (!aligned(c->table, 4) || !aligned(c->lens, 4) || !aligned(c->refs, 4) || !aligned(c->status, 4))
    return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// The calls that count or move pages: a page is one block of memory in each plane.
fa_status check_pages(const fakv_cache* c) {
  const fa_status st = check_cache(c);
  if (st != FA_OK) return st;
  if (!c->refs) return FA_ERR_INVALID_ARG;
  const long long head = c->D, row = (long long)c->HKV * c->D;
  const bool tokens_first = c->head_stride == head && c->token_stride == row;
  const bool heads_first = c->token_stride == head && c->head_stride == (long long)c->page_size * c->D;
  if (!tokens_first && !heads_first) return FA_ERR_UNSUPPORTED;
  const long long page = row * c->page_size;
  if (page * esize(c->dtype) > (1ll << 30)) return FA_ERR_UNSUPPORTED;
  if (c->page_stride < page) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_rope(const fakv_rope* r, int D) {
  if (!r || !r->freqs || (r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->mscale))
    return FA_ERR_INVALID_ARG;
  if (r->rotary_dim < 2 || r->rotary_dim > D || r->rotary_dim % 2 != 0) return FA_ERR_INVALID_ARG;
  return aligned(r->freqs, 8) ? FA_OK : FA_ERR_ALIGNMENT;
}

// (dtype: of q, k and v)
fa_status check_tokens(const fakv_cache* c, fa_dtype dtype, const fakv_tokens* p, const int* cu, const int* slots) {
  if (!p || p->B < 0 || p->B > MAX_SEQS || p->T < 0 || p->T > (1 << 30) || p->H < 0 || p->H > 65535)
    return FA_ERR_INVALID_ARG;
  if (p->plane < 0 || p->plane >= c->planes) return FA_ERR_INVALID_ARG;
  if (p->H % c->HKV != 0 || p->H / c->HKV > 128) return FA_ERR_INVALID_ARG;
  if ((double)p->T * p->H > 1073741824.0) return FA_ERR_INVALID_ARG;
  const int es = esize(dtype);
  for (long long s : {p->q_token, p->q_head, p->k_token, p->k_head, p->v_token, p->v_head})
    if (!stride_ok(s, es) || (double)p->T * s * es > MAX_BYTES) return FA_ERR_INVALID_ARG;
  if (p->B > 0 && p->T > 0 && !cu) return FA_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || !aligned(slots, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

fa_status check_append(const void* q, const void* k, const void* v, const void* q_out, fa_dtype dtype, int D,
                       const fakv_tokens* p) {
  const int es = esize(dtype);
  if (!k || !v || (p->H > 0 && (!q || !q_out))) return FA_ERR_INVALID_ARG;
  if (!aligned(k, es) || !aligned(v, es) || (p->H > 0 && (!aligned(q, es) || !aligned(q_out, es))))
    return FA_ERR_ALIGNMENT;
  // in place: contiguous (the stride of one token or one head is no matter)
  if (p->H > 0 && q == q_out && ((p->H > 1 && p->q_head != D) || (p->T > 1 && p->q_token != (long long)p->H * D)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_attend(const fakv_tokens* p) {
  if (p->H < 1 || !dtype_ok(p->out_dtype)) return FA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f && std::isfinite(p->scale * LOG2E))) return FA_ERR_INVALID_ARG;
  if ((p->causal != 0 && p->causal != 1) || p->window < 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_attend_rows(const void* q, const void* O, const void* LSE, fa_dtype dtype, const fakv_tokens* p) {
  for (const void* x : {q, O, LSE}) {
    if (!x) return FA_ERR_INVALID_ARG;
    if (!aligned(x, 16)) return FA_ERR_ALIGNMENT;
  }
  const int es = esize(dtype);
  return p->q_token * es % 16 != 0 || p->q_head * es % 16 != 0 ? FA_ERR_ALIGNMENT : FA_OK;
}

bool quant_ok(int page_size, int D, int bits, int group) {
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return false;
  if (D < 16 || D % 16 != 0 || D > 128 || (bits != 4 && bits != 8)) return false;
  return group == D || (D == 128 && group == 64);
}
// bytes of a token of one head
int quant_token(int D, int bits, int group) { return 16 * q_chunks(D, bits) + 4 * (D / group); }

// A cache in 4 or 8 bits as the page calls see it: one of 32-bit words, a token of one head as wide as
// its codes and params. (A block is page_size such tokens; which of its bytes are whose is no matter.)
fa_status check_qcache(const fakv_qcache* c, fakv_cache* pages) {
  if (!c || !dtype_ok(c->dtype)) return FA_ERR_INVALID_ARG;
  if (c->planes < 1 || c->num_pages < 1 || c->HKV < 1 || c->D < 1 || c->max_slots < 1 || c->max_pages < 1 ||
      c->page_size < 1 || c->group < 1)
    return FA_ERR_INVALID_ARG;
  if (!quant_ok(c->page_size, c->D, c->bits, c->group)) return FA_ERR_UNSUPPORTED;
  const int token = quant_token(c->D, c->bits, c->group);
  if (c->head_stride < token * c->page_size) return FA_ERR_INVALID_ARG;
  for (long long s : {c->page_stride, c->head_stride, c->planes > 1 ? c->plane_stride : 0})
    if (s % 16 != 0) return FA_ERR_ALIGNMENT;
  fakv_cache v = {};
  v.K = c->K;
  v.V = c->V;
  v.table = c->table;
  v.lens = c->lens;
  v.refs = c->refs;
  v.status = c->status;
  v.plane_stride = c->plane_stride / 4;
  v.page_stride = c->page_stride / 4;
  v.token_stride = 16;  // (tokens have none: what check_cache accepts)
  v.head_stride = c->head_stride / 4;
  v.table_stride = c->table_stride;
  v.planes = c->planes;
  v.num_pages = c->num_pages;
  v.page_size = c->page_size;
  v.HKV = c->HKV;
  v.D = 16;
  v.max_slots = c->max_slots;
  v.max_pages = c->max_pages;
  v.dtype = FA_F32;
  const fa_status st = check_cache(&v);
  if (st != FA_OK) return st;
  v.D = token / 4;
  *pages = v;
  return FA_OK;
}

// The calls that count or move pages
fa_status check_qpages(const fakv_qcache* c, fakv_cache* pages) {
  const fa_status st = check_qcache(c, pages);
  if (st != FA_OK) return st;
  if (!c->refs) return FA_ERR_INVALID_ARG;
  const long long block = (long long)quant_token(c->D, c->bits, c->group) * c->page_size;
  if (c->HKV > 1 && c->head_stride != block) return FA_ERR_UNSUPPORTED;
  if (block * c->HKV > (1ll << 30)) return FA_ERR_UNSUPPORTED;
  return c->page_stride < block * c->HKV ? FA_ERR_INVALID_ARG : FA_OK;
}

QCache qcache_of(const fakv_qcache& c, const fakv_cache& pages, int plane) {
  QCache q;
  q.c = pages;
  q.c.D = c.D;
  q.c.dtype = c.dtype;
  q.K = static_cast<uint8_t*>(c.K) + plane * (c.planes > 1 ? c.plane_stride : 0);
  q.V = static_cast<uint8_t*>(c.V) + plane * (c.planes > 1 ? c.plane_stride : 0);
  q.page = c.page_stride;
  q.head = c.head_stride;
  q.bits = c.bits;
  q.chunks = q_chunks(c.D, c.bits);
  q.groups = c.D / c.group;
  q.params = c.page_size * q.chunks * 16;
  return q;
}

fa_status grow(const fakv_cache& c, const int* slots, const int* add, int n, fa_stream_t stream) {
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!slots || !add) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(add, 4)) return FA_ERR_ALIGNMENT;
  return launch_grow(c, slots, add, n, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fork(const fakv_cache& c, const int* src, const int* dst, int n, fa_stream_t stream) {
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if ((long long)n * c.max_pages > (1ll << 31)) return FA_ERR_INVALID_ARG;  // rows held meanwhile
  if (n == 0) return FA_OK;
  if (!src || !dst) return FA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return FA_ERR_ALIGNMENT;
  return launch_fork(c, src, dst, n, reinterpret_cast<cudaStream_t>(stream));
}

fa_status release(const fakv_cache& c, const int* slots, const int* keep, int n, fa_stream_t stream) {
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!slots) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(keep, 4)) return FA_ERR_ALIGNMENT;
  return launch_free(c, slots, keep, n, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace kv
}  // namespace fa

using namespace fa;
using namespace fa::kv;

extern "C" {

FA_API fa_status fakv_rope_freqs(int rotary_dim, double base, const fakv_scaling* scaling,
                                 unsigned long long* freqs, float* mscale) {
  const fakv_scaling plain = {};
  const fakv_scaling& s = scaling ? *scaling : plain;
  if (!freqs || !mscale || rotary_dim < 2 || rotary_dim > 128 || rotary_dim % 2 != 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(base) && base > 1.0)) return FA_ERR_INVALID_ARG;
  if (s.kind < FAKV_PLAIN || s.kind > FAKV_YARN) return FA_ERR_INVALID_ARG;
  if (s.kind != FAKV_PLAIN && !(std::isfinite(s.factor) && s.factor > 0)) return FA_ERR_INVALID_ARG;
  if (s.kind == FAKV_NTK && rotary_dim == 2) return FA_ERR_INVALID_ARG;
  if ((s.kind == FAKV_BANDS || s.kind == FAKV_YARN) && !(std::isfinite(s.original) && s.original > 0))
    return FA_ERR_INVALID_ARG;
  if (s.kind == FAKV_BANDS && !(std::isfinite(s.low) && std::isfinite(s.high) && s.low < s.high))
    return FA_ERR_INVALID_ARG;
  if (s.kind == FAKV_YARN &&
      !(std::isfinite(s.beta_fast) && s.beta_slow > 0 && s.beta_fast > s.beta_slow))
    return FA_ERR_INVALID_ARG;
  const double pi2 = 6.283185307179586476925286766559, r = rotary_dim;
  if (s.kind == FAKV_NTK) base *= std::pow(s.factor, r / (r - 2));
  if (!(std::isfinite(base) && base > 1.0)) return FA_ERR_INVALID_ARG;
  double a = 0, b = 0;
  if (s.kind == FAKV_YARN) {
    auto e = [&](double beta) { return r * std::log(s.original / (pi2 * beta)) / (2 * std::log(base)); };
    a = std::fmax(std::floor(e(s.beta_fast)), 0);
    b = std::fmin(std::ceil(e(s.beta_slow)), r - 1);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (s.kind == FAKV_LINEAR) f /= s.factor;
    if (s.kind == FAKV_BANDS) {
      const double t = (s.original * f / pi2 - s.low) / (s.high - s.low);
      const double w = std::fmin(std::fmax(t, 0), 1);
      f *= (1 - w) / s.factor + w;
    }
    if (s.kind == FAKV_YARN) {
      const double g = std::fmin(std::fmax((i - a) / std::fmax(b - a, 0.001), 0), 1);
      f *= g / s.factor + 1 - g;
    }
    double turns = f / pi2;  // whole turns do not count
    turns -= std::floor(turns);
    const double x = turns * 18446744073709551616.0;  // 2^64, exact
    freqs[i] = x >= 18446744073709551616.0 ? 0 : (unsigned long long)x;
  }
  *mscale = s.kind == FAKV_YARN && s.factor > 1 ? (float)(0.1 * std::log(s.factor) + 1.0) : 1.f;
  return FA_OK;
}

FA_API fa_status fakv_rope_apply(const void* q, const void* k, void* q_out, void* k_out,
                                 const void* positions, const fakv_rope* rope,
                                 const fakv_rope_params* p, fa_stream_t stream) {
  if (!p || !dtype_ok(p->dtype) || p->T < 0 || p->T > (1 << 30) || p->H < 1 || p->HKV < 0 || p->D < 1)
    return FA_ERR_INVALID_ARG;
  if (p->H > 65535 || p->HKV > 65535) return FA_ERR_INVALID_ARG;
  if ((p->positions_64 != 0 && p->positions_64 != 1) || (p->inverse != 0 && p->inverse != 1))
    return FA_ERR_INVALID_ARG;
  if (p->D % 16 != 0 || p->D > 128) return FA_ERR_UNSUPPORTED;
  fa_status st = check_rope(rope, p->D);
  if (st != FA_OK) return st;
  const int es = esize(p->dtype);
  for (long long s : {p->q_token, p->q_head, p->k_token, p->k_head, p->qo_token, p->qo_head, p->ko_token, p->ko_head})
    if (!stride_ok(s, es) || (double)p->T * s * es > MAX_BYTES) return FA_ERR_INVALID_ARG;
  if (p->T == 0) return FA_OK;
  if (!q || !q_out || !positions || (p->HKV > 0 && (!k || !k_out))) return FA_ERR_INVALID_ARG;
  if (!aligned(q, es) || !aligned(q_out, es) || !aligned(positions, p->positions_64 ? 8 : 4)) return FA_ERR_ALIGNMENT;
  if (p->HKV > 0 && (!aligned(k, es) || !aligned(k_out, es))) return FA_ERR_ALIGNMENT;
  // in place: element for element
  if (q == q_out && (p->q_token != p->qo_token || p->q_head != p->qo_head)) return FA_ERR_INVALID_ARG;
  if (p->HKV > 0 && k == k_out && (p->k_token != p->ko_token || p->k_head != p->ko_head)) return FA_ERR_INVALID_ARG;
  // output rows that overlap would be written, and in place read, by several threads at once
  if ((p->H > 1 && p->qo_head < p->D) || (p->T > 1 && p->qo_token < p->D)) return FA_ERR_INVALID_ARG;
  if ((p->HKV > 1 && p->ko_head < p->D) || (p->HKV > 0 && p->T > 1 && p->ko_token < p->D)) return FA_ERR_INVALID_ARG;
  return launch_rope(q, k, q_out, k_out, positions, *rope, *p, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_append(const void* q, const void* k, const void* v, void* q_out,
                             const int* cu, const int* slots, const fakv_rope* rope,
                             const fakv_cache* cache, const fakv_tokens* p, fa_stream_t stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  st = check_tokens(cache, cache->dtype, p, cu, slots);
  if (st != FA_OK) return st;
  if (rope && (st = check_rope(rope, cache->D)) != FA_OK) return st;
  if (p->B == 0 || p->T == 0) return FA_OK;
  if ((st = check_append(q, k, v, q_out, cache->dtype, cache->D, p)) != FA_OK) return st;
  return launch_append(q, k, v, q_out, cu, slots, rope, *cache, *p, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_attend(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                             const fakv_cache* cache, const fakv_tokens* p, fa_stream_t stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  st = check_tokens(cache, cache->dtype, p, cu, slots);
  if (st != FA_OK) return st;
  if ((st = check_attend(p)) != FA_OK) return st;
  if (p->B == 0 || p->T == 0) return FA_OK;
  if ((st = check_attend_rows(q, O, LSE, cache->dtype, p)) != FA_OK) return st;
  fakv_tokens t = *p;
  if (t.window >= cache->max_pages * cache->page_size) t.window = 0;  // hides nothing
  // Above 16 rows per sequence and kv head (on average: the lengths are on the device) tensor-core
  // tiles, if the copy engine can take the tensors' strides. 16 sequences of 8192 tokens (32
  // query heads on 8 of 128): 16 rows 65 us by rows, 84 by tiles; 32 rows 104 and 77. An average
  // serves a mixed batch badly on both sides: 256 sequences decoding and a chunk, over 4096
  // tokens each, take 890 us by rows just below the limit (a chunk of 700), 748 in two calls;
  // over 1024, 274 by tiles just above it (1100) and 238.
  if (cache->dtype == FA_BF16 && (long long)t.T * (t.H / cache->HKV) > 16ll * t.B) {
    st = launch_attend_tiles(q, O, LSE, cu, slots, *cache, t, reinterpret_cast<cudaStream_t>(stream));
    if (st != FA_ERR_UNSUPPORTED) return st;
  }
  return launch_attend_rows(q, O, LSE, cu, slots, *cache, t, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_grow(const fakv_cache* cache, const int* slots, const int* add, int n,
                           fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  return st != FA_OK ? st : grow(*cache, slots, add, n, stream);
}

FA_API fa_status fakv_fork(const fakv_cache* cache, const int* src, const int* dst, int n,
                           fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  return st != FA_OK ? st : kv::fork(*cache, src, dst, n, stream);
}

FA_API fa_status fakv_free(const fakv_cache* cache, const int* slots, const int* keep, int n,
                           fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  return st != FA_OK ? st : release(*cache, slots, keep, n, stream);
}

FA_API fa_status fakv_compact(const fakv_cache* cache, fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  if (st != FA_OK) return st;
  return launch_compact(*cache, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ the cache in 4 or 8 bits
FA_API long long fakv_qblock_bytes(int page_size, int D, int bits, int group) {
  return quant_ok(page_size, D, bits, group) ? (long long)page_size * quant_token(D, bits, group) : 0;
}

FA_API fa_status fakv_qappend(const void* q, const void* k, const void* v, void* q_out,
                              const int* cu, const int* slots, const fakv_rope* rope,
                              const fakv_qcache* cache, const fakv_tokens* p, fa_stream_t stream) {
  fakv_cache pages;
  fa_status st = check_qcache(cache, &pages);
  if (st != FA_OK) return st;
  if ((st = check_tokens(&pages, cache->dtype, p, cu, slots)) != FA_OK) return st;
  if (rope && (st = check_rope(rope, cache->D)) != FA_OK) return st;
  if (p->B == 0 || p->T == 0) return FA_OK;
  if ((st = check_append(q, k, v, q_out, cache->dtype, cache->D, p)) != FA_OK) return st;
  return launch_qappend(q, k, v, q_out, cu, slots, rope, qcache_of(*cache, pages, p->plane), *p,
                        reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_qread(void* K_out, void* V_out, const int* cu, const int* slots,
                            const int* first, const fakv_qcache* cache, const fakv_tokens* p,
                            fa_stream_t stream) {
  fakv_cache pages;
  fa_status st = check_qcache(cache, &pages);
  if (st != FA_OK) return st;
  if (!p) return FA_ERR_INVALID_ARG;
  fakv_tokens t = {};
  t.B = p->B;
  t.T = p->T;
  t.plane = p->plane;
  t.out_dtype = p->out_dtype;
  if ((st = check_tokens(&pages, cache->dtype, &t, cu, slots)) != FA_OK) return st;
  if (!dtype_ok(t.out_dtype) || (double)t.T * cache->HKV > 1073741824.0) return FA_ERR_INVALID_ARG;
  if (!aligned(first, 4)) return FA_ERR_ALIGNMENT;
  if (t.B == 0 || t.T == 0) return FA_OK;
  if (!K_out || !V_out) return FA_ERR_INVALID_ARG;
  if (!aligned(K_out, 16) || !aligned(V_out, 16)) return FA_ERR_ALIGNMENT;
  const uintptr_t k = reinterpret_cast<uintptr_t>(K_out), v = reinterpret_cast<uintptr_t>(V_out);
  if ((k > v ? k - v : v - k) < (uintptr_t)t.T * cache->HKV * cache->D * esize(t.out_dtype)) return FA_ERR_INVALID_ARG;
  return launch_qread(K_out, V_out, cu, slots, first, qcache_of(*cache, pages, t.plane), t,
                      reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_qattend(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                              const fakv_qcache* cache, const fakv_tokens* p, fa_stream_t stream) {
  fakv_cache pages;
  fa_status st = check_qcache(cache, &pages);
  if (st != FA_OK) return st;
  if ((st = check_tokens(&pages, cache->dtype, p, cu, slots)) != FA_OK) return st;
  if ((st = check_attend(p)) != FA_OK) return st;
  if (p->B == 0 || p->T == 0) return FA_OK;
  if ((st = check_attend_rows(q, O, LSE, cache->dtype, p)) != FA_OK) return st;
  fakv_tokens t = *p;
  if (t.window >= cache->max_pages * cache->page_size) t.window = 0;  // hides nothing
  // Above this many rows per sequence and kv head (on average) tensor-core tiles, whose time hardly depends on how many
  // there are, where kv_qrows.cu makes numbers of all codes again for every 16. 8 kv heads, us (rows, tiles):
  //                                 4 bits: 32 rows  48 rows   64 rows   80 rows     8 bits: 48 rows   64 rows   80 rows
  //   16 sequences of up to 8192       74,  95  108,  98  134, 101  163, 100            118, 121  141, 123  174, 122
  //   64 of up to 2048                 85, 114  116, 117  148, 118  179, 121            123, 135  154, 138  189, 140
  //   4 of up to 65536                121, 172  172, 172  223, 172  269, 175            176, 207  232, 208  275, 211
  //   one of 16384                     28,  36   34,  36   40,  36   44,  36             35,  41   40,  41   46,  42
  //   16 of up to 8192, D 64           51,  92   70,  92   88,  95  107,  94             73,  85   90,  88  112,  87
  // One short sequence is better served by rows for longer (4096 tokens: up to 100), but lengths are on the device.
  const long long limit = cache->D > 64 ? 48 : 64;
  if (cache->dtype == FA_BF16 && (long long)t.T * (t.H / cache->HKV) > limit * t.B) {
    st = launch_qattend_tiles(q, O, LSE, cu, slots, qcache_of(*cache, pages, p->plane), t,
                              reinterpret_cast<cudaStream_t>(stream));
    if (st != FA_ERR_UNSUPPORTED) return st;
  }
  return launch_qattend_rows(q, O, LSE, cu, slots, qcache_of(*cache, pages, p->plane), t,
                             reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_qgrow(const fakv_qcache* cache, const int* slots, const int* add, int n,
                            fa_stream_t stream) {
  fakv_cache pages;
  const fa_status st = check_qpages(cache, &pages);
  return st != FA_OK ? st : grow(pages, slots, add, n, stream);
}

FA_API fa_status fakv_qfork(const fakv_qcache* cache, const int* src, const int* dst, int n,
                            fa_stream_t stream) {
  fakv_cache pages;
  const fa_status st = check_qpages(cache, &pages);
  return st != FA_OK ? st : kv::fork(pages, src, dst, n, stream);
}

FA_API fa_status fakv_qfree(const fakv_qcache* cache, const int* slots, const int* keep, int n,
                            fa_stream_t stream) {
  fakv_cache pages;
  const fa_status st = check_qpages(cache, &pages);
  return st != FA_OK ? st : release(pages, slots, keep, n, stream);
}

FA_API fa_status fakv_qcompact(const fakv_qcache* cache, fa_stream_t stream) {
  fakv_cache pages;
  const fa_status st = check_qpages(cache, &pages);
  return st != FA_OK ? st : launch_compact(pages, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
