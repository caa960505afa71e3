/*
 * fakv.h -- C ABI of libfa.so for served and trained models' positions and key / value
 * caches: rotary positions, a paged cache, attention of new tokens over it, and the
 * cache's pages (sharing, growing, freeing, compacting); and the same for a cache held in 4 or
 * 8 bits. It uses fa.h's types, status
 * codes, streams and ownership rules; fa_timing_* and fa_device_status cover its kernels too.
 *
 * The cache. Keys and values live in pages of `page_size` tokens. A slot is one
 * sequence: row s of `table` holds the page numbers of its tokens in order, lens[s] its
 * length in tokens. refs[p] counts the rows that hold page p (0: free), so sequences
 * with a common beginning may share pages. A row holds the pages of its lens[s] tokens:
 * entries past them are -1, or are not counted on by grow, fork and free (grow writes over
 * them), so a length is lowered by fakv_free, which releases what is no longer needed. All of it is device memory that the caller
 * owns, and every call reads lengths, tables and counts on the device: a step's calls
 * (grow, append, attend) can be captured into a CUDA graph once and replayed while the
 * lengths move on. Calls on one cache must be ordered (one stream, or events).
 *
 *   page p, token t, kv head h, column d of K in plane l is
 *     K[l * plane_stride + p * page_stride + t * token_stride + h * head_stride + d]
 *   and the same for V (elements of `dtype`; d runs without gaps). Planes are what
 *   shares one table: the layers of a model.
 *
 * A call's new tokens are rows of q (and k, v): sequence b of the call has the rows
 * cu[b] .. cu[b + 1] - 1 (cu: B + 1 non-decreasing int32 from 0 to at most T; attend does
 * nothing with one that decreases) and is slot slots[b] (slots NULL: slot b; attend may
 * name a slot for several sequences). Lengths count the new tokens: row i of a sequence with n
 * new tokens has position lens[slot] - n + i. Rows from cu[B] on belong to no sequence:
 * their outputs are not written, and no output depends on what they hold, but they may
 * be read.
 *
 * What only the device can see is checked there: a slot outside [0, max_slots), a page
 * number outside [0, num_pages) where a token should be, a length beyond the row. Such
 * an entry is left out (keys read as zeros, tokens not written; in the page calls its
 * slot's length, row and counts stay as they were) and a bit is set in `*status`, which
 * the caller reads and clears. No access leaves the arrays described.
 * A wait inside a kernel that ran out (fa.h) is no bit of it: fa_device_status tells, and
 * outputs of the call may then be unwritten.
 *
 * Every call checks its arguments, enqueues on `stream` and returns. Temporary buffers come
 * stream-ordered from the library's pool, so calls on different streams, and graphs, do not
 * share them. A call may be captured once one call has run on the device outside a capture.
 */
#ifndef FAKV_H_
#define FAKV_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  FAKV_NO_PAGES = 1,   /* grow: fewer free pages than asked for; the entry was not served */
  FAKV_BAD_SLOT = 2,   /* a slot outside [0, max_slots) */
  FAKV_REPEATED = 4,   /* a slot named twice in one list: the first one counts */
  FAKV_ROW_FULL = 8,   /* grow: the row's max_pages pages do not suffice; not served */
  FAKV_BAD_PAGE = 16,  /* a table entry outside [0, num_pages) where a token should be */
  FAKV_BAD_LENGTH = 32 /* a length below 0, above max_pages * page_size or, in append, below the
                          new tokens; a cu that decreases; a negative add or keep */
};

typedef struct {
  void* K;                 /* 16-byte aligned */
  void* V;
  int* table;              /* [max_slots] rows of max_pages, table_stride apart; -1: no page */
  int* lens;               /* [max_slots] */
  int* refs;               /* [num_pages] */
  int* status;             /* one word, or NULL */
  long long plane_stride;  /* elements; each stride but the planes' of one plane is a */
  long long page_stride;   /* positive multiple of 16 bytes */
  long long token_stride;
  long long head_stride;
  long long table_stride;  /* >= max_pages */
  int planes;              /* >= 1 */
  int num_pages;           /* >= 1 */
  int page_size;           /* a power of two, 8 .. 1024 */
  int HKV;
  int D;                   /* a multiple of 16, 16 .. 128 */
  int max_slots;
  int max_pages;           /* pages in a row of the table; max_pages * page_size <= 2^30 */
  fa_dtype dtype;
} fakv_cache;

/* ---- rotary positions
 * The first `rotary_dim` columns of a head are rotary_dim / 2 pairs: columns (i, i +
 * rotary_dim / 2) (half), or (2 i, 2 i + 1) (interleaved). At position p, pair i turns by
 * p f_i and is multiplied by mscale; the other columns pass unchanged.
 *   f_i = base^(-2 i / rotary_dim), then by `kind`:
 *   FAKV_LINEAR  f_i / factor
 *   FAKV_NTK     base * factor^(r / (r - 2)) in place of base (r = rotary_dim > 2)
 *   FAKV_BANDS   with t_i = original f_i / 2 pi (turns over the original context):
 *                f_i where t_i >= high, f_i / factor where t_i <= low, between them
 *                (1 - s) f_i / factor + s f_i with s = (t_i - low) / (high - low)
 *   FAKV_YARN    the ramp g_i = clamp((i - a) / (b - a), 0, 1) between a = floor(e(beta_fast))
 *                and b = ceil(e(beta_slow)), e(x) = r ln(original / 2 pi x) / (2 ln base),
 *                a >= 0, b <= r - 1 (b - a at least 0.001): g_i f_i / factor + (1 - g_i) f_i,
 *                and mscale = 0.1 ln(factor) + 1 (1 for a factor up to 1).
 * fakv_rope_freqs (host only) writes what the kernels read: f_i as a 64-bit fraction of
 * a turn, so that p f_i modulo a whole turn is one integer product, exact for any
 * position: far positions lose nothing. The caller copies freqs to the device once. */
typedef enum { FAKV_PLAIN = 0, FAKV_LINEAR = 1, FAKV_NTK = 2, FAKV_BANDS = 3, FAKV_YARN = 4 } fakv_scaling_kind;

typedef struct {
  fakv_scaling_kind kind;
  double factor;    /* > 0 (all but PLAIN) */
  double low, high; /* BANDS: low < high */
  double original;  /* BANDS, YARN: > 0 */
  double beta_fast, beta_slow; /* YARN: beta_fast > beta_slow > 0 */
} fakv_scaling;

typedef struct {
  const unsigned long long* freqs; /* device, [rotary_dim / 2] */
  int rotary_dim;                  /* even, 2 .. D */
  int interleaved;                 /* 0: half, 1: interleaved */
  float mscale;
} fakv_rope;

FA_API fa_status fakv_rope_freqs(int rotary_dim, double base, const fakv_scaling* scaling,
                                 unsigned long long* freqs, float* mscale);

/* Rows of q [T, H, D] and k [T, HKV, D] (element strides per token and head, D without
 * gaps) turned by their positions, into q_out and k_out, which are the inputs themselves
 * (with the inputs' strides) or do not overlap them; rows of an output do not overlap. HKV = 0: no k. positions [T] int32,
 * or int64 with positions_64 = 1; any sign. inverse = 1 turns the other way: the gradient
 * of the rotation (mscale included). fp32 arithmetic, one rounding on store. */
typedef struct {
  int T, H, HKV, D;
  fa_dtype dtype;
  int positions_64, inverse;
  long long q_token, q_head, k_token, k_head;             /* element strides of the inputs */
  long long qo_token, qo_head, ko_token, ko_head;         /* and of the outputs */
} fakv_rope_params;

FA_API fa_status fakv_rope_apply(const void* q, const void* k, void* q_out, void* k_out,
                                 const void* positions, const fakv_rope* rope,
                                 const fakv_rope_params* p, fa_stream_t stream);

/* ---- the cache's tokens */
typedef struct {
  int B;                 /* sequences in the call, 0 .. 16384 */
  int T;                 /* rows of q, k, v */
  int H;                 /* query heads: a multiple of the cache's HKV, at most 128 HKV and 65535
                            (append: 0 for no q) */
  int plane;             /* the cache's plane */
  long long q_token, q_head;   /* element strides of q, multiples of 16 bytes (attend) */
  long long k_token, k_head;   /* append: of k */
  long long v_token, v_head;   /* append: of v */
  float scale;           /* attend: finite (times log2 e too), > 0 */
  int causal, window;    /* attend: key j visible to position p iff (!causal || j <= p) and
                            (window == 0 || j >= p - window + 1) */
  fa_dtype out_dtype;    /* attend: dtype of O */
} fakv_tokens;

/* k and v [T, HKV, D] written to their tokens' places, k turned by its positions first
 * where `rope` is given, and q [T, H, D] turned likewise into q_out [T, H, D] (contiguous;
 * copied where rope is NULL). q_out does not overlap the inputs, or is q itself if that is
 * contiguous. Inputs in the cache's dtype. A slot named for two sequences has two tokens for
 * a place: which of them stays is not defined. With a cu that decreases (a status bit) a row
 * may be taken for another sequence's; only places of that sequence's new tokens are then
 * written. One launch. */
FA_API fa_status fakv_append(const void* q, const void* k, const void* v, void* q_out,
                             const int* cu, const int* slots, const fakv_rope* rope,
                             const fakv_cache* cache, const fakv_tokens* p, fa_stream_t stream);

/* O [T, H, D] = softmax(scale q K^T + mask) V over the tokens of each row's sequence, LSE
 * [T, H] (natural log) fp32; contiguous. Query head h reads kv head h / (H / HKV). q in the
 * cache's dtype. A row that sees no key gets O = 0, LSE = -inf. K and V within a
 * sequence's length must be finite, K below 2^127 and V below 2^80 in size (probabilities of
 * up to 2^8 times V are summed over the keys in fp32); page memory past it may hold anything.
 * NaN or infinity in a row of q makes that row's O and LSE NaN and no other's. fp32 caches
 * use three tf32 products per GEMM (about 22 significant bits); bf16 caches bf16 products
 * with fp32 sums, the probabilities in bf16: two terms (2^-16) where O is fp32 or there are few
 * rows, one (2^-8, about a bf16 O's own rounding) where there are many and O is bf16. Sums
 * over keys that are split between CTAs are joined in a fixed order: results do not
 * depend on timing. A batch is served by one kernel, chosen by the average T / B of rows to a
 * sequence (what the host knows: rows from cu[B] on count). So a few long chunks among
 * hundreds of decoding sequences are better given calls of their own, and T is better the
 * step's own row count than a buffer's: padding a decoding step above 16 rows per sequence and
 * kv head takes the kernel of chunks, with a bf16 O's one-term probabilities. */
FA_API fa_status fakv_attend(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                             const fakv_cache* cache, const fakv_tokens* p, fa_stream_t stream);

/* ---- the cache's pages. `slots`, `src`, `dst`, `add`, `keep`: device int32 [n]. */

/* Room for add[i] >= 0 more tokens in slots[i], and lens grown by it. New pages are the
 * lowest free ones, in the order of the list. A last page that has room but is shared
 * (refs > 1 when the call starts) is first replaced by a copy, in every plane. An entry
 * is not served (its length stays) if its row is too short, if the last page that its new
 * tokens begin in is missing or, with the entries before it, it needs more pages than were
 * free. Its step is then to be left out too: an append that counts on the pages would take the
 * slot's last tokens for the new ones and write over them. */
FA_API fa_status fakv_grow(const fakv_cache* cache, const int* slots, const int* add, int n,
                           fa_stream_t stream);

/* Slots dst[i] become copies of slots src[i], sharing their pages; what dst[i] held is
 * released. All at once: sources are read as they were before the call, so a list may
 * exchange or reorder slots. n * max_pages <= 2^31; above 32 entries, or 256 pages to a row,
 * the rows are held meanwhile in 4 n max_pages bytes of scratch. An entry of a row that
 * names no page is copied as it is, counted nowhere (BAD_PAGE). */
FA_API fa_status fakv_fork(const fakv_cache* cache, const int* src, const int* dst, int n,
                           fa_stream_t stream);

/* Slots cut to min(lens, keep[i]) tokens (keep NULL: 0), pages no longer needed released. */
FA_API fa_status fakv_free(const fakv_cache* cache, const int* slots, const int* keep, int n,
                           fa_stream_t stream);

/* With L pages in use, the used pages numbered L and above move, in order, to the free
 * numbers below L (in every plane), and all rows (over their whole width, whatever their
 * lengths) and counts follow: pages 0 .. L - 1 are then the used ones. */
FA_API fa_status fakv_compact(const fakv_cache* cache, fa_stream_t stream);

/* ---- the cache in 4 or 8 bits
 * A cache like the one above whose pages hold codes. Of a token's K (or V) row of one head, each
 * group of `group` columns x has a scale s and an offset z, both bf16, and a code per column:
 *
 *   z = the largest bf16 <= min x         s = the smallest bf16 >= (max x - z) / (2^bits - 1)
 *   c = (x - z) / s, to the nearest integer (ties to even), at most 2^bits - 1    (s = 0: c = 0)
 *
 * (the differences and quotients are fp32, rounded to nearest), and stands for s c + z: at most
 * s / 2 from x, where s is (max x - min x) / (2^bits - 1) but for the roundings of s and z
 * (2^-7 of it, and 2^-7 |min x| / (2^bits - 1)). A group that holds NaN, infinity or a value of
 * 2^126 or more has no such scale: its s and z are NaN, and so is all that it stands for.
 *
 * Memory, in bytes. Page p, head h in plane l is a block at K + l * plane_stride + p * page_stride
 * + h * head_stride, of page_size * (16 chunks + 4 groups) bytes with chunks = ceil(D * bits / 128)
 * and groups = D / group:
 *   K codes [page_size / 8][chunks][8 tokens][16]: chunk k of a token has its columns
 *           k * 128 / bits and on, in order, lowest bits first (columns from D on: 0)
 *   V codes [page_size / 8][chunks][4][32]: the same for two tokens, 2 i and 2 i + 1, side by
 *           side: in turn 16 bits (4 bits a code) or 8 bits (8) of each
 *   params  [page_size][groups]: s in the low, z in the high 16 bits of a 32-bit word
 * Slots, tables, lengths, counts, status, ownership, ordering, capture and what is refused are as
 * above. */
typedef struct {
  void* K;                 /* 16-byte aligned */
  void* V;
  int* table;              /* [max_slots] rows of max_pages, table_stride apart; -1: no page */
  int* lens;               /* [max_slots] */
  int* refs;               /* [num_pages] */
  int* status;             /* one word, or NULL */
  long long plane_stride;  /* bytes; each but the planes' of one plane is a positive multiple */
  long long page_stride;   /* of 16, and head_stride at least a block */
  long long head_stride;
  long long table_stride;  /* >= max_pages */
  int planes;              /* >= 1 */
  int num_pages;           /* >= 1 */
  int page_size;           /* a power of two, 8 .. 1024 */
  int HKV;
  int D;                   /* a multiple of 16, 16 .. 128 */
  int max_slots;
  int max_pages;           /* max_pages * page_size <= 2^30 */
  int bits;                /* 4 or 8 */
  int group;               /* D, or 64 where D is 128 */
  fa_dtype dtype;          /* of q, k and v */
} fakv_qcache;

/* Bytes of a block (a page of one head), or 0 for sizes that no cache has. */
FA_API long long fakv_qblock_bytes(int page_size, int D, int bits, int group);

/* fakv_append into such a cache: k turned by its positions where `rope` is given, in fp32 and
 * without a rounding before its codes are formed; v; and q into q_out as fakv_append does. (A slot named
 * for two sequences: a place's codes may be of one token and its scale of the other.) */
FA_API fa_status fakv_qappend(const void* q, const void* k, const void* v, void* q_out,
                              const int* cu, const int* slots, const fakv_rope* rope,
                              const fakv_qcache* cache, const fakv_tokens* p, fa_stream_t stream);

/* What the cache stands for, s c + z in fp32 with one rounding on store, as contiguous
 * K_out, V_out [T, HKV, D] of out_dtype (16-byte aligned, not overlapping): row i of sequence b is position
 * first[b] + i of its slot (first NULL: the slot's last tokens, position lens - n + i). Rows of a
 * sequence whose token does not exist (a bad slot, a position outside [0, lens), no page) are
 * zeros and set the status bit; rows from cu[B] on are not written. Of `p` the call reads B, T,
 * plane and out_dtype. One launch. */
FA_API fa_status fakv_qread(void* K_out, void* V_out, const int* cu, const int* slots,
                            const int* first, const fakv_qcache* cache, const fakv_tokens* p,
                            fa_stream_t stream);

/* fakv_attend over what such a cache stands for, s c + z; K and V below 2^80 in size (what is below
 * 2^-100 may count for less than it is). Precision, beyond that of the codes:
 *   few rows to a sequence, and every fp32 q: q times a power of two in fp16 (a bf16 q exactly but for
 *     what is 2^-28 of its row's largest value; an fp32 q in two terms, 2^-22), codes exactly, scales and
 *     offsets in fp32, fp32 sums; a probability times its key's scale in fp16, one term (2^-11) where O is
 *     bf16, two (2^-22) where it is fp32
 *   many rows (bf16 q): K and q as above (scales of K to 2^-21 of the key's largest value), so that LSE
 *     is too; V to 2^-11 of the value and of its two parts, codes times scale and offset, and a
 *     probability to 2^-11: of an fp32 O too, whose last bits are better had from fp32 queries or from
 *     fewer rows to a call
 * Products of a probability and a key's V are taken against the largest V of the keys that the row has
 * gone through so far: those 2^-14 of it and smaller lose bits, those below 2^-30 count for nothing (an
 * O that is made of them alone, beside far larger V, is good to that, and not to 2^-11 of itself). Keys
 * that a row does not see have no part in it, whatever their size (many rows: V up to 2^3 times as large
 * as that of a key next to it that the row does see may be what its products are taken against).
 * Scores (times log2 e) are below 2^127 in size; of 2^20 and more they are rounded to 24 bits each before
 * the largest is taken off.
 * NaN or infinity in a row of q makes that row's O and LSE NaN and no other's. A key that stands for NaN makes
 * the rows that see it NaN (K: O and LSE; V: their O in the group's columns, and where there are many
 * rows all of O, and LSE) and no other. Which kernel is chosen, T and a batch of both kinds: as for fakv_attend,
 * but with 48 rows per sequence and kv head (64 where D is at most 64) as the limit. */
FA_API fa_status fakv_qattend(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                              const fakv_qcache* cache, const fakv_tokens* p, fa_stream_t stream);

/* The page calls. */
FA_API fa_status fakv_qgrow(const fakv_qcache* cache, const int* slots, const int* add, int n,
                            fa_stream_t stream);
FA_API fa_status fakv_qfork(const fakv_qcache* cache, const int* src, const int* dst, int n,
                            fa_stream_t stream);
FA_API fa_status fakv_qfree(const fakv_qcache* cache, const int* slots, const int* keep, int n,
                            fa_stream_t stream);
FA_API fa_status fakv_qcompact(const fakv_qcache* cache, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FAKV_H_ */
