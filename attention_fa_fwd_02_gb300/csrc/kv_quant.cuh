// kv_quant.cuh -- the cache in 4 or 8 bits (include/fakv.h has its format): where things lie,
// and codes to numbers.
//
// A code becomes a bf16 number by setting bits, not by a conversion: bf16 has seven bits behind
// its point, so the nibble n in the lowest four of them of 128.0 (0x4300) is 128 + n, in the
// highest four of 16.0 (0x4180) 16 + n, of 256.0 (0x4380) 256 + 16 n. One shift and one
// three-input logic instruction make two of them, in the two halves of a register.
#pragma once
#include "kv_common.cuh"

namespace fa {
namespace kv {

struct QCache {
  fakv_cache c;         // slots, table, lengths, counts, status; sizes (what K and V hold is not in it)
  uint8_t* K;           // of the call's plane
  uint8_t* V;
  long long page, head; // strides in bytes
  int bits, chunks, groups;
  int params;           // offset of the params in a block
};

inline int q_chunks(int D, int bits) { return (D * bits + 127) / 128; }

// of codes: 16-byte chunk k of token t (both of a block)
__host__ __device__ __forceinline__ int q_code_at(int chunks, int t, int k) {
  return ((t >> 3) * chunks + k) * 128 + (t & 7) * 16;
}

__device__ __forceinline__ float q_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float q_offset(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Nibbles R and R + 4 of a word as two bf16: Q_BIAS[R] + n
template <int R>
__device__ __forceinline__ uint32_t q_pair(uint32_t w) {
  if constexpr (R == 0) return (w & 0x000f000fu) | 0x43004300u;
  else return ((w >> (4 * R - 3)) & 0x00780078u) | 0x41804180u;
}
__host__ __device__ constexpr float q_bias(int r) { return r == 0 ? 128.f : 16.f; }
// The same nibbles as 256 + 16 n (R > 0)
template <int R>
__device__ __forceinline__ uint32_t q_pair16(uint32_t w) {
  static_assert(R > 0, "needs a shift");
  return ((w >> (4 * R - 3)) & 0x00780078u) | 0x43804380u;
}

__device__ __forceinline__ uint32_t add_bf2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
// -x twice (x a bf16 number)
__host__ __device__ constexpr uint32_t q_minus(int x) {
  return x == 24 ? 0xc1c0c1c0u : x == 136 ? 0xc308c308u : x == 512 ? 0xc400c400u : /* 400 */ 0xc3c8c3c8u;
}

// Centred codes, n - 8 or c - 128: with the codes' mean near zero their sums lose nothing to a
// constant that is many times as large as what is summed up.
template <int R>
__device__ __forceinline__ uint32_t q_centred4(uint32_t w) {  // nibbles R and R + 4
  return add_bf2(q_pair<R>(w), q_minus(R == 0 ? 136 : 24));
}
template <int J>
__device__ __forceinline__ uint32_t q_centred8(uint32_t w) {  // bytes J and J + 2
  constexpr int LOW = 2 * J, HIGH = 2 * J + 1;
  // (every step exact: 256 + 16 h - 512 or - 400 has at most five significant bits)
  return add_bf2(add_bf2(q_pair16<HIGH>(w), q_minus(J == 0 ? 512 : 400)), q_pair<LOW>(w));
}
template <int BITS, int J>
__device__ __forceinline__ uint32_t q_centred(uint32_t w) {
  if constexpr (BITS == 4) return q_centred4<J>(w);
  else return q_centred8<J>(w);
}

fa_status launch_qappend(const void* q, const void* k, const void* v, void* qo, const int* cu, const int* slots,
                         const fakv_rope* r, const QCache& c, const fakv_tokens& p, cudaStream_t s);
fa_status launch_qread(void* K, void* V, const int* cu, const int* slots, const int* first, const QCache& c,
                       const fakv_tokens& p, cudaStream_t s);
fa_status launch_qattend_rows(const void* q, void* O, float* LSE, const int* cu, const int* slots, const QCache& c,
                              const fakv_tokens& p, cudaStream_t s);

}  // namespace kv
}  // namespace fa
