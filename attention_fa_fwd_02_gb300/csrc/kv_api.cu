// kv_api.cu -- the extern "C" boundary of include/fakv.h: argument checks and dispatch.
#include <cmath>
#include <initializer_list>
#include "kv_common.cuh"

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

fa_status check_tokens(const fakv_cache* c, const fakv_tokens* p, const int* cu, const int* slots) {
  if (!p || p->B < 0 || p->B > MAX_SEQS || p->T < 0 || p->T > (1 << 30) || p->H < 0 || p->H > 65535)
    return FA_ERR_INVALID_ARG;
  if (p->plane < 0 || p->plane >= c->planes) return FA_ERR_INVALID_ARG;
  if (p->H % c->HKV != 0 || p->H / c->HKV > 128) return FA_ERR_INVALID_ARG;
  if ((double)p->T * p->H > 1073741824.0) return FA_ERR_INVALID_ARG;
  const int es = esize(c->dtype);
  for (long long s : {p->q_token, p->q_head, p->k_token, p->k_head, p->v_token, p->v_head})
    if (!stride_ok(s, es) || (double)p->T * s * es > MAX_BYTES) return FA_ERR_INVALID_ARG;
  if (p->B > 0 && p->T > 0 && !cu) return FA_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || !aligned(slots, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
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
  st = check_tokens(cache, p, cu, slots);
  if (st != FA_OK) return st;
  if (rope && (st = check_rope(rope, cache->D)) != FA_OK) return st;
  if (p->B == 0 || p->T == 0) return FA_OK;
  const int es = esize(cache->dtype);
  if (!k || !v || (p->H > 0 && (!q || !q_out))) return FA_ERR_INVALID_ARG;
  if (!aligned(k, es) || !aligned(v, es) || (p->H > 0 && (!aligned(q, es) || !aligned(q_out, es))))
    return FA_ERR_ALIGNMENT;
  // in place: contiguous (the stride of one token or one head is no matter)
  if (p->H > 0 && q == q_out &&
      ((p->H > 1 && p->q_head != cache->D) || (p->T > 1 && p->q_token != (long long)p->H * cache->D)))
    return FA_ERR_INVALID_ARG;
  return launch_append(q, k, v, q_out, cu, slots, rope, *cache, *p, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_attend(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                             const fakv_cache* cache, const fakv_tokens* p, fa_stream_t stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  st = check_tokens(cache, p, cu, slots);
  if (st != FA_OK) return st;
  if (p->H < 1 || !dtype_ok(p->out_dtype)) return FA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f && std::isfinite(p->scale * LOG2E))) return FA_ERR_INVALID_ARG;
  if ((p->causal != 0 && p->causal != 1) || p->window < 0) return FA_ERR_INVALID_ARG;
  if (p->B == 0 || p->T == 0) return FA_OK;
  for (const void* x : {q, (const void*)O, (const void*)LSE}) {
    if (!x) return FA_ERR_INVALID_ARG;
    if (!aligned(x, 16)) return FA_ERR_ALIGNMENT;
  }
  const int es = esize(cache->dtype);
  if (p->q_token * es % 16 != 0 || p->q_head * es % 16 != 0) return FA_ERR_ALIGNMENT;
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
  if (st != FA_OK) return st;
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!slots || !add) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(add, 4)) return FA_ERR_ALIGNMENT;
  return launch_grow(*cache, slots, add, n, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_fork(const fakv_cache* cache, const int* src, const int* dst, int n,
                           fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  if (st != FA_OK) return st;
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if ((long long)n * cache->max_pages > (1ll << 31)) return FA_ERR_INVALID_ARG;  // rows held meanwhile
  if (n == 0) return FA_OK;
  if (!src || !dst) return FA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return FA_ERR_ALIGNMENT;
  return launch_fork(*cache, src, dst, n, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_free(const fakv_cache* cache, const int* slots, const int* keep, int n,
                           fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  if (st != FA_OK) return st;
  if (n < 0 || n > MAX_SEQS) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!slots) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(keep, 4)) return FA_ERR_ALIGNMENT;
  return launch_free(*cache, slots, keep, n, reinterpret_cast<cudaStream_t>(stream));
}

FA_API fa_status fakv_compact(const fakv_cache* cache, fa_stream_t stream) {
  const fa_status st = check_pages(cache);
  if (st != FA_OK) return st;
  return launch_compact(*cache, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
