// kv_quant.cu -- new tokens quantised into the cache in 4 or 8 bits, and the cache read back.
//
// A row (a token of one head of q, k or v) is taken by four lanes, which hold its columns eight at
// a time: lane `quad` has columns 32 w + 8 quad .. + 7 of every block w of 32. So eight columns are
// one 16-byte load (bf16), a 4-bit code word or two 8-bit ones; a group's minimum and maximum are
// a few operations in the lane and two shuffles; and a warp's eight rows, the same head of eight
// tokens where a block has as many, meet in whole 128-byte lines of codes.
//
// Rows are turned as in kv_rope.cu: cos and sin once per token and pair, in shared memory. Codes
// are formed from the fp32 result of the turn, with IEEE differences and quotients, so that they
// are those of the definition whatever else changes here.
//
// Measured (append and the reading back of what it wrote, two calls; device, data in L2): a step of 48 sequences, 32 heads
// on 8 of 128, 11.2 us, four dependent look-ups (cu, slot and length, table, row) each; ragged chunks of up to 1024 tokens for 8
// sequences in 8 bits 27.8 us (36 cold; bytes at the copy rate 10): the arithmetic of the codes, one block's share of rows
// after another. A division a code took 32.5, rows asked for after their places 14.0 for the step; three blocks an SM
// (spilled registers) and shorter spans were slower. Reading 8 sequences of up to 16384 into fp32 69 us (floor 46),
// 4.6 TB/s, nearly all of it stores; with half sectors to a store 78.
#include <cmath>
#include "kv_quant.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int THREADS = 256;
constexpr int ROWS = 8;    // of a warp
constexpr int SPAN = THREADS / 8;  // tokens of a block at most (eight lanes look each up)
constexpr float LARGE = 8.507059173023462e37f;  // 2^126

struct MoveArgs {
  QCache q;
  // append: rows in and (q) out; read: rows out
  const void* src[3];
  void* dst[3];
  long long token[3], head[3];  // strides of src (append)
  int H, T, B, D, shift;
  int span, span_shift, per;  // tokens of a block (and their log2); rows of a token in it (gridDim.y parts)
  int rot, interleaved, wide;
  const unsigned long long* freqs;
  float mscale;
  const int* cu;
  const int* slots;
  const int* first;
  int out_bf16;
};

template <typename E>
__device__ __forceinline__ float load1(const E* p);
template <>
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load1(const float* p) { return *p; }

template <typename E>
__device__ __forceinline__ void unpack8(const uint4 (&v)[sizeof(E) / 2], float (&x)[8]) {
  if constexpr (sizeof(E) == 2) {
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(v[i].x);
      x[4 * i + 1] = __uint_as_float(v[i].y);
      x[4 * i + 2] = __uint_as_float(v[i].z);
      x[4 * i + 3] = __uint_as_float(v[i].w);
    }
  }
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// the largest bf16 <= x (finite, below 2^126 in size), as fp32
__device__ __forceinline__ float down(float x) {
  const int i = __float_as_int(x), cut = i & (int)0xffff0000;
  return __int_as_float(i < 0 && i != cut ? cut + 0x10000 : cut);
}

// Scale and offset of values between lo and hi
struct Grid {
  float s, z;
};
__device__ __forceinline__ Grid grid_of(float lo, float hi, float steps, bool fine) {
  Grid g;
  g.z = down(lo);
  g.s = -down(-__fdiv_rn(__fsub_rn(hi, g.z), steps));
  if (!fine) g.s = g.z = __int_as_float(0x7fff0000);  // NaN
  return g;
}
// The codes of eight columns: quotients rounded to integers. A product with 1 / s (exact, as the fused operations take
// it) is off from the quotient by less than 2^-14 (of up to 256: 2^-23 of it and of 1 / s), so it rounds to the same
// integer unless it lies that near to the middle between two; there, one value in some thousands, the quotients of its eight
// columns are formed. The integers stand in the low bits of 1.5 * 2^23 and more.
__device__ __forceinline__ void codes_of(const float (&x)[8], const Grid& g, float inv, uint32_t (&code)[8]) {
  constexpr float MAGIC = 12582912.f;
  bool near = false;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const float d = __fsub_rn(x[n], g.z), y = __fmaf_rn(d, inv, MAGIC);
    const float off = __fmaf_rn(d, inv, -__fsub_rn(y, MAGIC));
    near |= !(fabsf(off) <= 0.5f - 0x1p-13f);  // (NaN too: s may be 0, or too small for 1 / s)
    code[n] = __float_as_uint(y);
  }
  if (near) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
      code[n] = g.s > 0.f ? __float_as_uint(__fadd_rn(rintf(__fdiv_rn(__fsub_rn(x[n], g.z), g.s)), MAGIC)) : 0u;
  }
}

// Place of the block's tokens in a page: page number and token, or page -1 (no such token); live: the row
// belongs to a sequence; its position there.
struct Places {
  int page[SPAN], at[SPAN], live[SPAN];
  long long pos[SPAN];
};

// The places of rows t0 .. t0 + tokens - 1, eight lanes to a row: its sequence is the last b with cu[b] <= t, eight
// probes to a round (cu is probed inside [0, B] whatever it holds).
template <bool READ>
__device__ __forceinline__ void find_places(const MoveArgs& a, int t0, int tokens, Places& sh) {
  const fakv_cache& c = a.q.c;
  const int k = threadIdx.x / 8, sub = threadIdx.x & 7, t = t0 + min(k, tokens - 1);
  if (threadIdx.x / 32 * 4 >= tokens) return;  // (whole warps)
  int lo = 0, n = a.B;  // the answer lies in [lo, lo + n)
  const int end = a.cu[a.B];
  bool live = t < end;
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + 7) / 8;
    const bool below = sub * step < n && a.cu[lo + sub * step] <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, below) >> (threadIdx.x & 24) & 0xffu);
    const int first = max(hits - 1, 0) * step;
    n = min(step, n - first);
    lo += first;
  }
  live = live && a.cu[lo] <= t;
  int page = -1;
  long long pos = 0;
  if (live && k < tokens) {
    const Seq s = load_seq(c, a.cu, a.slots, lo, a.T);
    pos = READ && a.first ? (long long)a.first[lo] + (t - s.row0) : (long long)s.len - s.n + (t - s.row0);
    if (s.slot >= 0 && pos >= 0 && pos < s.len) page = page_of(c, s.slot, (int)pos, a.shift);
    else if (s.slot >= 0) raise(c.status, FAKV_BAD_LENGTH);
  }
  if (k < tokens && sub == 0) {
    sh.page[k] = page;
    sh.at[k] = (int)pos & (c.page_size - 1);
    sh.live[k] = live;
    sh.pos[k] = pos;
  }
}

// a decreasing cu, looked for by one block (its warps but the first)
__device__ __forceinline__ void check_cu(const MoveArgs& a) {
  if (blockIdx.x != 0 || blockIdx.y != 0 || threadIdx.x < 32) return;
  bool falls = false;
  for (int b = threadIdx.x - 32; b < a.B; b += THREADS - 32) falls |= a.cu[b + 1] < a.cu[b];
  if (falls) raise(a.q.c.status, FAKV_BAD_LENGTH);
}

template <typename E, int BITS, int NW>  // NW: blocks of 32 columns at most
__global__ void __launch_bounds__(THREADS, 2) qappend_kernel(const __grid_constant__ MoveArgs a) {
  extern __shared__ float2 cs[];  // [tokens][pairs]
  __shared__ Places sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3;
  const int t0 = blockIdx.x * a.span, tokens = min(a.span, a.T - t0);
  const int pairs = a.rot / 2, HKV = a.q.c.HKV;
  const int heads = a.H + 2 * HKV;  // of a token: q's, k's, v's
  const int h0 = blockIdx.y * a.per, mine = min(a.per, heads - h0);
  check_cu(a);
  // Row r of the block: head h of token k, the lane's blocks of columns of it and (half pairs) of its pairs' other halves.
  // The first ones are on their way while the places are found.
  constexpr int PARTS = sizeof(E) / 2;  // 16-byte pieces of eight columns
  struct Raw {
    uint4 x[NW][PARTS], y[NW][PARTS];
  };
  auto load = [&](int r, Raw& v) {
    const int k = r & (a.span - 1), h = h0 + (r >> a.span_shift);
    if (!a.wide || k >= tokens || h >= h0 + mine) return;
    const int which = h < a.H ? 0 : h < a.H + HKV ? 1 : 2;
    const int head = h - (which == 0 ? 0 : which == 1 ? a.H : a.H + HKV);
    const E* const row = static_cast<const E*>(a.src[which]) + (t0 + k) * a.token[which] + head * a.head[which];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c0 = w * 32 + quad * 8;
      if (c0 >= a.D) continue;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) v.x[w][i] = reinterpret_cast<const uint4*>(row + c0)[i];
      if (which < 2 && c0 < a.rot && !a.interleaved) {
        const E* const other = row + (c0 >= pairs ? c0 - pairs : c0 + pairs);
#pragma unroll
        for (int i = 0; i < PARTS; ++i) v.y[w][i] = reinterpret_cast<const uint4*>(other)[i];
      }
    }
  };
  Raw raw;
  load(warp * ROWS + lane / 4, raw);
  find_places<false>(a, t0, tokens, sh);
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * pairs; i += THREADS) {
    const float2 v = turn(sh.pos[i / pairs], a.freqs[i % pairs]);
    cs[i] = make_float2(v.x * a.mscale, v.y * a.mscale);
  }
  __syncthreads();
  // (all lanes of a warp take part in its shuffles)
  for (int r0 = warp * ROWS; r0 < mine * a.span; r0 += THREADS / 32 * ROWS) {
    const int r = r0 + lane / 4;
    if (r0 != warp * ROWS) load(r, raw);
    const int k = r & (a.span - 1), h = h0 + (r >> a.span_shift);
    const bool in = k < tokens && h < h0 + mine;
    const int which = h < a.H ? 0 : h < a.H + HKV ? 1 : 2;
    const int head = h - (which == 0 ? 0 : which == 1 ? a.H : a.H + HKV);
    const E* const row = static_cast<const E*>(a.src[which]) + (in ? (t0 + k) * a.token[which] + head * a.head[which] : 0);
    const bool turned = which < 2;
    float x[NW][8];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c0 = w * 32 + quad * 8;
#pragma unroll
      for (int n = 0; n < 8; ++n) x[w][n] = 0.f;
      if (!in || c0 >= a.D) continue;
      const float2* const turns = cs + k * pairs;
      if (a.wide) {
        unpack8<E>(raw.x[w], x[w]);
        if (turned && c0 < a.rot) {
          if (a.interleaved) {
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
              const float2 q = turns[(c0 + n) / 2];
              const float u = x[w][n], v = x[w][n + 1];
              x[w][n] = __fmaf_rn(-v, q.y, __fmul_rn(u, q.x));
              x[w][n + 1] = __fmaf_rn(u, q.y, __fmul_rn(v, q.x));
            }
          } else {
            const bool second = c0 >= pairs;
            float y[8];
            unpack8<E>(raw.y[w], y);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float2 q = turns[(second ? c0 - pairs : c0) + n];
              x[w][n] = second ? __fmaf_rn(y[n], q.y, __fmul_rn(x[w][n], q.x))
                               : __fmaf_rn(-y[n], q.y, __fmul_rn(x[w][n], q.x));
            }
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int c = c0 + n;
          x[w][n] = load1(row + c);
          if (turned && c < a.rot) {
            const int i = a.interleaved ? c / 2 : c < pairs ? c : c - pairs;
            const bool second = a.interleaved ? c & 1 : c >= pairs;
            const float y = load1(row + (a.interleaved ? c ^ 1 : second ? c - pairs : c + pairs));
            const float2 q = turns[i];
            x[w][n] = second ? __fmaf_rn(y, q.y, __fmul_rn(x[w][n], q.x)) : __fmaf_rn(-y, q.y, __fmul_rn(x[w][n], q.x));
          }
        }
      }
    }
    __syncwarp();  // q_out may be q: the row's lanes have read each other's columns
    if (which == 0 && in && sh.live[k]) {
      E* const out = static_cast<E*>(a.dst[0]) + ((size_t)(t0 + k) * a.H + head) * a.D;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int c0 = w * 32 + quad * 8;
        if (c0 >= a.D) continue;
        if (a.wide) {
          store8(out + c0, x[w]);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            if constexpr (sizeof(E) == 2) out[c0 + n] = __float2bfloat16_rn(x[w][n]);
            else out[c0 + n] = x[w][n];
          }
        }
      }
    }
    if (!__any_sync(0xffffffffu, in && which > 0)) continue;
    // ---- minimum and maximum of blocks 0, 1 and of 2, 3: of the groups, or both of the whole head
    constexpr float steps = BITS == 4 ? 15.f : 255.f;
    float lo[2] = {INFINITY, INFINITY}, hi[2] = {-INFINITY, -INFINITY};
    float nil[2] = {0.f, 0.f};  // (NaN where a value is NaN or infinite: the minimum and maximum pass over NaN)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w * 32 + quad * 8 >= a.D) continue;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        lo[w / 2] = fminf(lo[w / 2], x[w][n]);
        hi[w / 2] = fmaxf(hi[w / 2], x[w][n]);
        nil[w / 2] = fmaf(x[w][n], 0.f, nil[w / 2]);
      }
    }
    if (a.q.groups == 1) {
      lo[0] = lo[1] = fminf(lo[0], lo[1]);
      hi[0] = hi[1] = fmaxf(hi[0], hi[1]);
      nil[0] = nil[1] = nil[0] + nil[1];
    }
    Grid g[2];
    float inv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], d));
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], d));
        nil[i] += __shfl_xor_sync(0xffffffffu, nil[i], d);
      }
      g[i] = grid_of(lo[i], hi[i], steps, nil[i] == 0.f && hi[i] < LARGE && lo[i] > -LARGE);
      inv[i] = __fdiv_rn(1.f, g[i].s);
    }
    // V's tokens lie in pairs: where the lanes four off have the pair's other one, each writes half of what both have
    const int k2 = k ^ 1;
    const bool paired = a.span > 1 && in && which == 2 && k2 < tokens && sh.page[k] >= 0 && sh.page[k2] == sh.page[k] &&
                        (sh.at[k] ^ 1) == sh.at[k2] && (sh.at[k] & 1) == (k & 1);
    const bool skip = which == 0 || !in || sh.page[k] < 0;
    uint8_t* const block = (which == 1 ? a.q.K : a.q.V) + (skip ? 0 : sh.page[k] * a.q.page + head * a.q.head);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const bool none = skip || (BITS == 4 ? w >= a.q.chunks : 2 * w + quad / 2 >= a.q.chunks);
      uint32_t code[8];
      codes_of(x[w], g[w / 2], inv[w / 2], code);
      if (w * 32 + quad * 8 >= a.D) {
#pragma unroll
        for (int n = 0; n < 8; ++n) code[n] = 0u;
      }
      if constexpr (BITS == 4) {
        // (bytes of columns 0, 2, 4, 6 and of 1, 3, 5, 7)
        const uint32_t e = __byte_perm(__byte_perm(code[0], code[2], 0x0040), __byte_perm(code[4], code[6], 0x0040), 0x5410);
        const uint32_t d = __byte_perm(__byte_perm(code[1], code[3], 0x0040), __byte_perm(code[5], code[7], 0x0040), 0x5410);
        const uint32_t v = e | d << 4;
        const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 4);
        if (none) continue;
        if (paired) {
          // (the even token's lane the words' low halves, the odd one's their high ones)
          uint32_t* const to = reinterpret_cast<uint32_t*>(block + q_v_at(4, a.q.chunks, sh.at[k] & ~1, w, quad));
          if (k & 1) to[1] = __byte_perm(o, v, 0x7632);
          else to[0] = __byte_perm(v, o, 0x5410);
        } else if (which == 1) *reinterpret_cast<uint32_t*>(block + q_k_at(a.q.chunks, sh.at[k], w, quad)) = v;
        else q_v_store<4>(block + q_v_at(4, a.q.chunks, sh.at[k], w, quad), v);
      } else {
        const uint2 v = make_uint2(__byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410),
                                   __byte_perm(__byte_perm(code[4], code[5], 0x0040), __byte_perm(code[6], code[7], 0x0040), 0x5410));
        const int chunk = 2 * w + quad / 2, word = quad % 2 * 2;
        const uint32_t o = __shfl_xor_sync(0xffffffffu, k & 1 ? v.x : v.y, 4);
        if (none) continue;
        if (paired) {
          // (the even token's lane the first words, the odd one's the second)
          const uint32_t e = k & 1 ? o : v.x, d = k & 1 ? v.y : o;
          *reinterpret_cast<uint2*>(block + q_v_at(8, a.q.chunks, sh.at[k] & ~1, chunk, word + (k & 1))) =
              make_uint2(__byte_perm(e, d, 0x5140), __byte_perm(e, d, 0x7362));
        } else if (which == 1) {
          *reinterpret_cast<uint2*>(block + q_k_at(a.q.chunks, sh.at[k], chunk, word)) = v;
        } else {
          q_v_store<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word), v.x);
          q_v_store<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word + 1), v.y);
        }
      }
    }
    if (!skip && quad < a.q.groups) {
      const Grid& m = g[NW > 2 ? quad & 1 : 0];
      *reinterpret_cast<uint32_t*>(block + a.q.params + (sh.at[k] * a.q.groups + quad) * 4) =
          (__float_as_uint(m.s) >> 16) | (__float_as_uint(m.z) & 0xffff0000u);
    }
  }
}

template <typename E, int BITS, int NW>
__global__ void __launch_bounds__(THREADS) qread_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ Places sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3;
  const int t0 = blockIdx.x * a.span, tokens = min(a.span, a.T - t0);
  const int HKV = a.q.c.HKV, heads = 2 * HKV;
  const int h0 = blockIdx.y * a.per, mine = min(a.per, heads - h0);
  check_cu(a);
  find_places<true>(a, t0, tokens, sh);
  __syncthreads();
  // A lane's columns of block w in two pieces of four: side by side (bf16: one 16-byte store) or 16 columns apart, so
  // that the row's four lanes fill 64 bytes with each store (8 sequences of up to 16384 tokens, 5 heads of 80: 69 us where halves of
  // sectors took 78).
  constexpr bool NEXT = sizeof(E) == 2;
  auto column = [&](int w, int i) { return w * 32 + (NEXT ? quad * 8 + i * 4 : i * 16 + quad * 4); };
  for (int r = warp * ROWS + lane / 4; r < mine * a.span; r += THREADS / 32 * ROWS) {
    const int k = r & (a.span - 1), h = h0 + (r >> a.span_shift);
    if (k >= tokens || !sh.live[k]) continue;
    const int which = h < HKV ? 0 : 1, head = h - which * HKV;
    const bool there = sh.page[k] >= 0;
    const uint8_t* const block = (which == 0 ? a.q.K : a.q.V) + (there ? sh.page[k] * a.q.page + head * a.q.head : 0);
    uint32_t code[NW][2], param[2] = {0u, 0u};  // (four codes in the low bits)
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = column(w, i), chunk = c * BITS / 128, word = c * BITS / 32 & 3;
        code[w][i] = 0u;
        if (!there || c >= a.D) continue;
        if constexpr (BITS == 4) {
          const uint8_t* const at = block + (which == 0 ? q_k_at(a.q.chunks, sh.at[k], chunk, word) + (c / 4 & 1) * 2
                                                        : q_v_at(4, a.q.chunks, sh.at[k], chunk, word) + (c / 4 & 1) * 4);
          code[w][i] = *reinterpret_cast<const uint16_t*>(at);
        } else {
          code[w][i] = which == 0 ? *reinterpret_cast<const uint32_t*>(block + q_k_at(a.q.chunks, sh.at[k], chunk, word))
                                  : q_v_load8(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word));
        }
      }
    if (there) {
      const uint32_t* const p = reinterpret_cast<const uint32_t*>(block + a.q.params + sh.at[k] * a.q.groups * 4);
      param[0] = p[0];
      param[1] = p[a.q.groups - 1];
    }
    E* const out = static_cast<E*>(a.dst[which]) + ((size_t)(t0 + k) * HKV + head) * a.D;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float s = q_scale(param[w / 2]), z = q_offset(param[w / 2]);
      float y[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) {  // (a code becomes a number in the low bits of 2^23)
        const uint32_t v = code[w][n / 4];
        const uint32_t c = BITS == 4 ? (v >> (4 * (n & 3))) & 15u : __byte_perm(v, 0u, 0x4440 | (n & 3));
        y[n] = fmaf(s, __uint_as_float(c | 0x4b000000u) - 8388608.f, z);
      }
      if constexpr (NEXT) {
        if (column(w, 0) < a.D) store8(out + column(w, 0), y);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (column(w, i) < a.D)
            *reinterpret_cast<float4*>(out + column(w, i)) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      }
    }
  }
}

// Tokens of a block: as many as leave every SM three blocks, and so few tokens are spread over their heads
void shape(MoveArgs& a, int heads, dim3* grid) {
  const int want = 3 * host::sm_count();
  a.span = SPAN;
  while (a.span > 1 && (a.T + a.span - 1) / a.span < want) a.span /= 2;
  const int blocks = (a.T + a.span - 1) / a.span;
  int parts = 1;
  // (a part keeps more than the eight rows of one warp; the block's other warps may have none, as in a step of few tokens)
  while (parts * blocks < want && heads * a.span > 2 * parts * ROWS) parts *= 2;
  a.per = (heads + parts - 1) / parts;
  a.span_shift = log2_of(a.span);
  *grid = dim3(blocks, (heads + a.per - 1) / a.per);
}

void fill(MoveArgs& a, const QCache& c, const fakv_tokens& p, const int* cu, const int* slots) {
  a.q = c;
  a.T = p.T;
  a.B = p.B;
  a.D = c.c.D;
  a.shift = log2_of(c.c.page_size);
  a.cu = cu;
  a.slots = slots;
}

template <typename E, int BITS>
fa_status append(MoveArgs& a, cudaStream_t s) {
  dim3 grid;
  shape(a, a.H + 2 * a.q.c.HKV, &grid);
  const size_t cs = (size_t)a.span * (a.rot / 2) * sizeof(float2);
  host::KernelTimer t("qappend", s);
  return launch(a.D <= 64 ? qappend_kernel<E, BITS, 2> : qappend_kernel<E, BITS, 4>, grid, THREADS, cs, s, a);
}

template <typename E, int BITS>
fa_status read(MoveArgs& a, cudaStream_t s) {
  dim3 grid;
  shape(a, 2 * a.q.c.HKV, &grid);
  host::KernelTimer t("qread", s);
  return launch(a.D <= 64 ? qread_kernel<E, BITS, 2> : qread_kernel<E, BITS, 4>, grid, THREADS, 0, s, a);
}

}  // namespace

fa_status launch_qappend(const void* q, const void* k, const void* v, void* qo, const int* cu, const int* slots,
                         const fakv_rope* r, const QCache& c, const fakv_tokens& p, cudaStream_t s) {
  MoveArgs a = {};
  fill(a, c, p, cu, slots);
  a.H = p.H;
  a.src[0] = q; a.src[1] = k; a.src[2] = v;
  a.dst[0] = qo;
  a.token[0] = p.q_token; a.token[1] = p.k_token; a.token[2] = p.v_token;
  a.head[0] = p.q_head; a.head[1] = p.k_head; a.head[2] = p.v_head;
  if (r) {
    a.rot = r->rotary_dim;
    a.interleaved = r->interleaved;
    a.freqs = r->freqs;
    a.mscale = r->mscale;
  }
  // 16-byte loads where strides, pointers and the pairs allow them
  const int ev = c.c.dtype == FA_BF16 ? 8 : 4;
  bool wide = a.rot % (a.interleaved ? 8 : 16) == 0;
  for (int i = p.H > 0 ? 0 : 1; i < 3; ++i)
    wide = wide && a.token[i] % ev == 0 && a.head[i] % ev == 0 && reinterpret_cast<uintptr_t>(a.src[i]) % 16 == 0;
  a.wide = wide && reinterpret_cast<uintptr_t>(qo) % 16 == 0;
  if (c.c.dtype == FA_BF16) return c.bits == 4 ? append<__nv_bfloat16, 4>(a, s) : append<__nv_bfloat16, 8>(a, s);
  return c.bits == 4 ? append<float, 4>(a, s) : append<float, 8>(a, s);
}

fa_status launch_qread(void* K, void* V, const int* cu, const int* slots, const int* first, const QCache& c,
                       const fakv_tokens& p, cudaStream_t s) {
  MoveArgs a = {};
  fill(a, c, p, cu, slots);
  a.dst[0] = K;
  a.dst[1] = V;
  a.first = first;
  if (p.out_dtype == FA_BF16) return c.bits == 4 ? read<__nv_bfloat16, 4>(a, s) : read<__nv_bfloat16, 8>(a, s);
  return c.bits == 4 ? read<float, 4>(a, s) : read<float, 8>(a, s);
}

}  // namespace kv
}  // namespace fa
