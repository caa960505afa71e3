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
#include <cmath>
#include "kv_quant.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int THREADS = 256;
constexpr int ROWS = 8;    // of a warp
constexpr int SPAN = 8;    // tokens of a block at most
constexpr float LARGE = 8.507059173023462e37f;  // 2^126

struct MoveArgs {
  QCache q;
  // append: rows in and (q) out; read: rows out
  const void* src[3];
  void* dst[3];
  long long token[3], head[3];  // strides of src (append)
  int H, T, B, D, shift;
  int span, per;  // tokens of a block; rows of a token in it (gridDim.y parts)
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

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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
__device__ __forceinline__ uint32_t code_of(float x, const Grid& g, float steps) {
  const float c = rintf(__fdiv_rn(__fsub_rn(x, g.z), g.s));
  return g.s > 0.f ? (uint32_t)fminf(fmaxf(c, 0.f), steps) : 0u;
}

// Place of the block's tokens in a page: page number and token, or page -1 (no such token); live: the row
// belongs to a sequence.
struct Places {
  int page[SPAN], at[SPAN], live[SPAN];
};

// Row t's position in its sequence and its place, by a warp
template <bool READ>
__device__ __forceinline__ long long find_place(const MoveArgs& a, int t, int k, Places& sh) {
  const fakv_cache& c = a.q.c;
  const int b = find_seq(a.cu, a.B, t);
  int page = -1;
  long long pos = 0;
  if (b >= 0) {
    const Seq s = load_seq(c, a.cu, a.slots, b, a.T);
    pos = READ && a.first ? (long long)a.first[b] + (t - s.row0) : (long long)s.len - s.n + (t - s.row0);
    if (s.slot >= 0 && pos >= 0 && pos < s.len) page = page_of(c, s.slot, (int)pos, a.shift);
    else if (s.slot >= 0) raise(c.status, FAKV_BAD_LENGTH);
  }
  if (ptx::lane_id() == 0) {
    sh.page[k] = page;
    sh.at[k] = (int)pos & (c.page_size - 1);
    sh.live[k] = b >= 0;
  }
  return pos;
}

// a decreasing cu, looked for by one block (its warps but the first)
__device__ __forceinline__ void check_cu(const MoveArgs& a) {
  if (blockIdx.x != 0 || blockIdx.y != 0 || threadIdx.x < 32) return;
  bool falls = false;
  for (int b = threadIdx.x - 32; b < a.B; b += THREADS - 32) falls |= a.cu[b + 1] < a.cu[b];
  if (falls) raise(a.q.c.status, FAKV_BAD_LENGTH);
}

template <typename E, int BITS, int NW>  // NW: blocks of 32 columns at most
__global__ void __launch_bounds__(THREADS) qappend_kernel(const __grid_constant__ MoveArgs a) {
  extern __shared__ float2 cs[];  // [tokens][pairs]
  __shared__ Places sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3;
  const int t0 = blockIdx.x * a.span, tokens = min(a.span, a.T - t0);
  const int pairs = a.rot / 2, HKV = a.q.c.HKV;
  const int heads = a.H + 2 * HKV;  // of a token: q's, k's, v's
  const int h0 = blockIdx.y * a.per, mine = min(a.per, heads - h0);
  check_cu(a);
  for (int k = warp; k < tokens; k += THREADS / 32) {
    const long long pos = find_place<false>(a, t0 + k, k, sh);
    for (int i = lane; i < pairs; i += 32) {
      const float2 v = turn(pos, a.freqs[i]);
      cs[k * pairs + i] = make_float2(v.x * a.mscale, v.y * a.mscale);
    }
  }
  __syncthreads();
  // (all lanes of a warp take part in its shuffles)
  for (int r0 = warp * ROWS; r0 < mine * a.span; r0 += THREADS / 32 * ROWS) {
    const int r = r0 + lane / 4;
    const int k = r % a.span, h = h0 + r / a.span;
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
        load8(row + c0, x[w]);
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
            load8(row + (second ? c0 - pairs : c0 + pairs), y);
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
    // ---- minimum and maximum of blocks 0, 1 and of 2, 3: of the groups, or both of the whole head
    constexpr float steps = BITS == 4 ? 15.f : 255.f;
    float lo[2] = {INFINITY, INFINITY}, hi[2] = {-INFINITY, -INFINITY};
    bool fine[2] = {true, true};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w * 32 + quad * 8 >= a.D) continue;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        lo[w / 2] = fminf(lo[w / 2], x[w][n]);
        hi[w / 2] = fmaxf(hi[w / 2], x[w][n]);
        fine[w / 2] = fine[w / 2] && fabsf(x[w][n]) < LARGE;
      }
    }
    if (a.q.groups == 1) {
      lo[0] = lo[1] = fminf(lo[0], lo[1]);
      hi[0] = hi[1] = fmaxf(hi[0], hi[1]);
      fine[0] = fine[1] = fine[0] && fine[1];
    }
    Grid g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], d));
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], d));
        fine[i] = __shfl_xor_sync(0xffffffffu, (int)fine[i], d) && fine[i];
      }
      g[i] = grid_of(lo[i], hi[i], steps, fine[i]);
    }
    if (which == 0 || !in || sh.page[k] < 0) continue;
    uint8_t* const block = (which == 1 ? a.q.K : a.q.V) + sh.page[k] * a.q.page + head * a.q.head;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (BITS == 4 ? w >= a.q.chunks : 2 * w + quad / 2 >= a.q.chunks) continue;
      uint32_t code[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) code[n] = w * 32 + quad * 8 < a.D ? code_of(x[w][n], g[w / 2], steps) : 0u;
      if constexpr (BITS == 4) {
        uint32_t v = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) v |= code[n] << (4 * n);
        if (which == 1) *reinterpret_cast<uint32_t*>(block + q_k_at(a.q.chunks, sh.at[k], w, quad)) = v;
        else q_v_store<4>(block + q_v_at(4, a.q.chunks, sh.at[k], w, quad), v);
      } else {
        uint2 v = make_uint2(0, 0);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          v.x |= code[n] << (8 * n);
          v.y |= code[4 + n] << (8 * n);
        }
        const int chunk = 2 * w + quad / 2, word = quad % 2 * 2;
        if (which == 1) {
          *reinterpret_cast<uint2*>(block + q_k_at(a.q.chunks, sh.at[k], chunk, word)) = v;
        } else {
          q_v_store<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word), v.x);
          q_v_store<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word + 1), v.y);
        }
      }
    }
    if (quad < a.q.groups) {
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
  for (int k = warp; k < tokens; k += THREADS / 32) find_place<true>(a, t0 + k, k, sh);
  __syncthreads();
  for (int r = warp * ROWS + lane / 4; r < mine * a.span; r += THREADS / 32 * ROWS) {
    const int k = r % a.span, h = h0 + r / a.span;
    if (k >= tokens || !sh.live[k]) continue;
    const int which = h < HKV ? 0 : 1, head = h - which * HKV;
    const bool there = sh.page[k] >= 0;
    const uint8_t* const block = (which == 0 ? a.q.K : a.q.V) + (there ? sh.page[k] * a.q.page + head * a.q.head : 0);
    uint2 code[NW];
    uint32_t param[2] = {0u, 0u};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      code[w] = make_uint2(0u, 0u);
      if (!there || w * 32 + quad * 8 >= a.D) continue;
      if constexpr (BITS == 4) {
        code[w].x = which == 0 ? *reinterpret_cast<const uint32_t*>(block + q_k_at(a.q.chunks, sh.at[k], w, quad))
                               : q_v_load<4>(block + q_v_at(4, a.q.chunks, sh.at[k], w, quad));
      } else {
        const int chunk = 2 * w + quad / 2, word = quad % 2 * 2;
        if (which == 0) {
          code[w] = *reinterpret_cast<const uint2*>(block + q_k_at(a.q.chunks, sh.at[k], chunk, word));
        } else {
          code[w].x = q_v_load<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word));
          code[w].y = q_v_load<8>(block + q_v_at(8, a.q.chunks, sh.at[k], chunk, word + 1));
        }
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
      const int c0 = w * 32 + quad * 8;
      if (c0 >= a.D) continue;
      const uint32_t p = param[w / 2];
      float y[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint32_t c = BITS == 4 ? (code[w].x >> (4 * n)) & 15u : ((n < 4 ? code[w].x : code[w].y) >> (8 * (n & 3))) & 255u;
        y[n] = fmaf(q_scale(p), (float)c, q_offset(p));
      }
      store8(out + c0, y);
    }
  }
}

// Tokens of a block: as many as leave every SM two blocks, and so few tokens are spread over their heads
void shape(MoveArgs& a, int heads, dim3* grid) {
  const int want = 2 * host::sm_count();
  a.span = SPAN;
  while (a.span > 1 && (a.T + a.span - 1) / a.span < want) a.span /= 2;
  const int blocks = (a.T + a.span - 1) / a.span;
  int parts = 1;
  // (a part has a warp's rows for each of its warps at least)
  while (parts * blocks < want && heads * a.span > 2 * parts * ROWS) parts *= 2;
  a.per = (heads + parts - 1) / parts;
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
