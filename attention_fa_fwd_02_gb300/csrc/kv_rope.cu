// kv_rope.cu -- rotary positions, and new tokens into the paged cache.
//
// Pair i of a head turns by the angle p f_i (mod 2 pi). The frequencies are 64-bit
// fractions of a turn, so p f_i mod 1 is the low word of one 64-bit product, exact for
// every position. Its nearest quarter turn is taken off in integers and the remainder (at
// most an eighth of a turn, 32 bits of it kept) goes through sincospif: cos and sin are
// good to fp32 rounding however far the position.
//
// Both operators are bound by the bytes of q, k, v, once in and once out. A unit is 2 EV
// columns of one head, two 16-byte accesses: the two halves of EV pairs, or 2 EV adjacent
// columns. A thread keeps one unit and takes it through UB tokens, so indices are found
// once and UB loads are on their way while the block forms the tokens' cos / sin, once for
// all heads, in shared memory (by itself a unit would need EV sincos per 32 bytes moved,
// more issue slots than the copy leaves). Measured: 8192 tokens of 32 + 8 heads of 128 in bf16
// 28.6 us, 168 MB at 5.9 TB/s, 32768 tokens 99 us, 6.8 TB/s (UB 2 or 8: 33, 41 us); one token
// 2.8 us. Append: 17000 tokens of 32 + 2 x 8 heads 74 us (floor 66); 4100 tokens 11.6 us with
// their 59 MB in L2 and 16.7 without (floor 8.7), where finding the tokens' pages (three
// dependent look-ups) and a last wave of blocks a third full show; a step of 48 tokens 4.2 us.
#include <cmath>
#include "kv_common.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int MAX_THREADS = 512;
constexpr int UB = 4;            // tokens per thread
constexpr int CS_BYTES = 16384;  // cos / sin of a block's tokens
constexpr int MAX_TOKENS = 64;   // per block

struct Stream {  // rows of one tensor
  const void* src;
  void* dst;
  long long s_token, s_head, d_token, d_head;
};

struct RopeArgs {
  Stream x[3];  // q, k, v
  int end[3];   // q: heads [0, end[0]), k: [end[0], end[1]), v: [end[1], end[2])
  int T;          // rows
  int lanes;      // threads per unit: tokens of a block side by side
  int deep;       // tokens per thread, 1 .. UB
  int rot, interleaved;
  int units;      // units of a head that are moved
  int per_token;  // units of a token
  const unsigned long long* freqs;
  float mscale, sign;
  const void* positions;
  int positions_64;
  // append
  const int* cu;
  const int* slots;
  int B, shift, plane;
  fakv_cache c;
};

template <typename E, int EV>
struct Chunk;  // EV elements: 16 bytes, or one element
template <>
struct Chunk<__nv_bfloat16, 8> { using V = uint4; };
template <>
struct Chunk<float, 4> { using V = uint4; };
template <>
struct Chunk<__nv_bfloat16, 1> { using V = uint16_t; };
template <>
struct Chunk<float, 1> { using V = uint32_t; };

template <typename E, int EV>
__device__ __forceinline__ void unpack(const typename Chunk<E, EV>::V& c, float (&f)[EV]) {
  if constexpr (EV == 1) {
    if constexpr (sizeof(E) == 2) f[0] = __uint_as_float((uint32_t)c << 16);
    else f[0] = __uint_as_float(c);
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(w[i]);
      }
    }
  }
}
template <typename E, int EV>
__device__ __forceinline__ typename Chunk<E, EV>::V pack(const float (&f)[EV]) {
  typename Chunk<E, EV>::V c;
  if constexpr (EV == 1) {
    if constexpr (sizeof(E) == 2) c = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    else c = __float_as_uint(f[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = __float_as_uint(f[i]);
      }
    }
    c.x = w[0]; c.y = w[1]; c.z = w[2]; c.w = w[3];
  }
  return c;
}

template <typename E, int EV, bool APPEND, bool ROPE>
__global__ void __launch_bounds__(MAX_THREADS, 2) rope_kernel(const __grid_constant__ RopeArgs a) {
  using V = typename Chunk<E, EV>::V;
  extern __shared__ float2 cs[];           // [tokens][pairs]
  __shared__ long long place[MAX_TOKENS];  // append: offset in the cache; -1: not written
  __shared__ int live[MAX_TOKENS];         // append: the row belongs to a sequence
  const int span = a.lanes * a.deep;       // tokens of a block
  const int t0 = blockIdx.x * span;
  const int tokens = min(span, a.T - t0);
  const int pairs = a.rot / 2;

  // this thread's unit: columns c0 .., c1 .. of one head (pair: its first pair, -1: copied)
  const int lane_t = a.lanes > 1 ? threadIdx.x / a.per_token : 0;
  const int u = a.lanes > 1 ? threadIdx.x - lane_t * a.per_token : blockIdx.y * blockDim.x + threadIdx.x;
  const bool any = u < a.per_token && lane_t < a.lanes;
  const int h = u / a.units, col = u - h * a.units;
  const int which = h < a.end[0] ? 0 : h < a.end[1] ? 1 : 2;
  const int head = h - (which ? a.end[which - 1] : 0);
  const bool turned = ROPE && col < pairs / EV;
  const int pair = turned && which < 2 ? col * EV : -1;
  const int c0 = turned && !a.interleaved ? col * EV : col * 2 * EV;
  const int c1 = turned && !a.interleaved ? c0 + pairs : c0 + EV;
  const Stream& x = a.x[which];
  V in[UB][2];
  {
    const E* p = static_cast<const E*>(x.src) + head * x.s_head;
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const int k = lane_t + i * a.lanes;
      if (any && i < a.deep && k < tokens) {
        const E* r = p + (t0 + k) * x.s_token;
        in[i][0] = *reinterpret_cast<const V*>(r + c0);
        in[i][1] = *reinterpret_cast<const V*>(r + c1);
      }
    }
  }

  if constexpr (APPEND) {
    // One block looks over the whole of cu (no row need lie where it decreases): its warps but the
    // first, whose look-ups for a token take longer.
    const int first = blockDim.x > 32 ? 32 : 0;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x >= first) {
      bool falls = false;
      for (int b = threadIdx.x - first; b < a.B; b += blockDim.x - first) falls |= a.cu[b + 1] < a.cu[b];
      if (falls) raise(a.c.status, FAKV_BAD_LENGTH);
    }
  }

  // positions, places, cos and sin of the block's tokens, a warp per token
  for (int k = threadIdx.x / 32; k < tokens; k += blockDim.x / 32) {
    const int t = t0 + k;
    long long pos = 0;
    if constexpr (APPEND) {
      const int b = find_seq(a.cu, a.B, t);
      long long at = -1;
      if (b >= 0) {
        const Seq s = load_seq(a.c, a.cu, a.slots, b, a.T);
        pos = (long long)s.len - s.n + (t - s.row0);
        if (s.slot >= 0 && pos >= 0 && pos < s.len) {
          const int page = page_of(a.c, s.slot, (int)pos, a.shift);
          if (page >= 0)
            at = a.plane * a.c.plane_stride + page * a.c.page_stride +
                 ((int)pos & (a.c.page_size - 1)) * a.c.token_stride;
        } else if (s.slot >= 0) {
          raise(a.c.status, FAKV_BAD_LENGTH);
        }
      }
      if (ptx::lane_id() == 0) { place[k] = at; live[k] = b >= 0; }
    } else {
      pos = a.positions_64 ? static_cast<const long long*>(a.positions)[t]
                           : static_cast<const int*>(a.positions)[t];
    }
    if constexpr (ROPE) {
      for (int i = ptx::lane_id(); i < pairs; i += 32) {
        const float2 v = turn(pos, a.freqs[i]);
        // (pair i = c EV + j at j (pairs / EV) + c: neighbouring units read neighbouring words)
        cs[k * pairs + (i % EV) * (pairs / EV) + i / EV] = make_float2(v.x * a.mscale, v.y * (a.mscale * a.sign));
      }
    }
  }
  __syncthreads();

  E* const out = static_cast<E*>(x.dst) + head * x.d_head;
#pragma unroll
  for (int i = 0; i < UB; ++i) {
    const int k = lane_t + i * a.lanes;
    if (!any || i >= a.deep || k >= tokens) continue;
    E* r;
    if (APPEND && which > 0) {
      if (place[k] < 0) continue;
      r = out + place[k];
    } else {
      if (APPEND && !live[k]) continue;
      r = out + (t0 + k) * x.d_token;
    }
    if (ROPE && pair >= 0) {
      float f[2][EV], y[2][EV];
      unpack<E, EV>(in[i][0], f[0]);
      unpack<E, EV>(in[i][1], f[1]);
      const float2* w = &cs[k * pairs + pair / EV];
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        // half: pair j is (f[0][j], f[1][j]); interleaved: columns 2 j, 2 j + 1
        const float2 q = w[j * (pairs / EV)];
        const float u_ = a.interleaved ? f[2 * j / EV][2 * j % EV] : f[0][j];
        const float v_ = a.interleaved ? f[(2 * j + 1) / EV][(2 * j + 1) % EV] : f[1][j];
        // (written out, so that wide and narrow units round alike)
        const float yu = __fmaf_rn(-v_, q.y, __fmul_rn(u_, q.x)), yv = __fmaf_rn(u_, q.y, __fmul_rn(v_, q.x));
        if (a.interleaved) { y[2 * j / EV][2 * j % EV] = yu; y[(2 * j + 1) / EV][(2 * j + 1) % EV] = yv; }
        else { y[0][j] = yu; y[1][j] = yv; }
      }
      in[i][0] = pack<E, EV>(y[0]);
      in[i][1] = pack<E, EV>(y[1]);
    }
    *reinterpret_cast<V*>(r + c0) = in[i][0];
    *reinterpret_cast<V*>(r + c1) = in[i][1];
  }
}

template <typename E, int EV, bool APPEND>
fa_status run(RopeArgs& a, const char* name, cudaStream_t s) {
  // A token's units side by side, in blocks of up to MAX_THREADS; where they are few,
  // several tokens side by side. Each thread takes UB tokens if that leaves every SM two
  // blocks, else one: few rows are spread over the SMs.
  a.per_token = a.end[2] * a.units;
  const int parts = (a.per_token + MAX_THREADS - 1) / MAX_THREADS;
  const int pairs = a.rot / 2;
  int most = MAX_TOKENS;
  if (pairs && CS_BYTES / 8 / pairs < most) most = CS_BYTES / 8 / pairs;
  a.lanes = 256 / a.per_token;
  if (a.lanes > most / UB) a.lanes = most / UB;
  if (a.lanes < 1) a.lanes = 1;
  a.deep = a.T >= 2 * UB * a.lanes * host::sm_count() ? UB : 1;
  const int threads = a.lanes > 1 ? a.lanes * a.per_token : (a.per_token + parts - 1) / parts;
  const int span = a.lanes * a.deep;
  const dim3 grid((a.T + span - 1) / span, parts), block((threads + 31) / 32 * 32);
  const size_t cs = (size_t)span * pairs * sizeof(float2);
  host::KernelTimer t(name, s);
  return launch(a.rot ? rope_kernel<E, EV, APPEND, true> : rope_kernel<E, EV, APPEND, false>, grid, block, cs, s, a);
}

template <bool APPEND>
fa_status dispatch(RopeArgs& a, int D, fa_dtype dtype, bool inplace, const char* name, cudaStream_t s) {
  // 16-byte chunks where the pairs, the strides and the pointers allow them
  const int ev = dtype == FA_BF16 ? 8 : 4, es = esize(dtype);
  bool wide = a.rot % (2 * ev) == 0;
  for (int i = 0; i < 3; ++i) {
    if (a.end[i] == (i ? a.end[i - 1] : 0)) continue;
    const Stream& x = a.x[i];
    for (long long v : {x.s_token, x.s_head, x.d_token, x.d_head}) wide = wide && v % ev == 0;
    wide = wide && (reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst)) % 16 == 0;
  }
  // in place the columns behind the pairs stay where they are
  a.units = (inplace ? a.rot : D) / (wide ? 2 * ev : 2);
  if (es == 2) return wide ? run<__nv_bfloat16, 8, APPEND>(a, name, s) : run<__nv_bfloat16, 1, APPEND>(a, name, s);
  return wide ? run<float, 4, APPEND>(a, name, s) : run<float, 1, APPEND>(a, name, s);
}

}  // namespace

fa_status launch_rope(const void* q, const void* k, void* qo, void* ko, const void* pos,
                      const fakv_rope& r, const fakv_rope_params& p, cudaStream_t s) {
  RopeArgs a = {};
  a.x[0] = {q, qo, p.q_token, p.q_head, p.qo_token, p.qo_head};
  a.x[1] = {k, ko, p.k_token, p.k_head, p.ko_token, p.ko_head};
  a.end[0] = p.H;
  a.end[1] = a.end[2] = p.H + p.HKV;
  a.T = p.T;
  a.rot = r.rotary_dim;
  a.interleaved = r.interleaved;
  a.freqs = r.freqs;
  a.mscale = r.mscale;
  a.sign = p.inverse ? -1.f : 1.f;
  a.positions = pos;
  a.positions_64 = p.positions_64;
  const bool inplace = (p.H == 0 || q == qo) && (p.HKV == 0 || k == ko);
  return dispatch<false>(a, p.D, p.dtype, inplace, "rope", s);
}

fa_status launch_append(const void* q, const void* k, const void* v, void* qo, const int* cu,
                        const int* slots, const fakv_rope* r, const fakv_cache& c,
                        const fakv_tokens& p, cudaStream_t s) {
  RopeArgs a = {};
  a.x[0] = {q, qo, p.q_token, p.q_head, (long long)p.H * c.D, c.D};
  a.x[1] = {k, c.K, p.k_token, p.k_head, c.token_stride, c.head_stride};
  a.x[2] = {v, c.V, p.v_token, p.v_head, c.token_stride, c.head_stride};
  a.end[0] = p.H;
  a.end[1] = p.H + c.HKV;
  a.end[2] = p.H + 2 * c.HKV;
  a.T = p.T;
  if (r) {
    a.rot = r->rotary_dim;
    a.interleaved = r->interleaved;
    a.freqs = r->freqs;
    a.mscale = r->mscale;
  }
  a.sign = 1.f;
  a.cu = cu;
  a.slots = slots;
  a.B = p.B;
  a.plane = p.plane;
  a.shift = log2_of(c.page_size);
  a.c = c;
  return dispatch<true>(a, c.D, c.dtype, false, "append", s);
}

}  // namespace kv
}  // namespace fa
