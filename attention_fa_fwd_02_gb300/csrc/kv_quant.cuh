// kv_quant.cuh -- the cache in 4 or 8 bits (include/fakv.h has its format): where things lie,
// and codes to numbers.
//
// A code becomes an fp16 number by setting bits, not by a conversion: fp16 has ten bits behind its
// point, so the low bits n of 1024.0 (0x6400) make 1024 + n. A byte is put there by one permute, two
// of them in the two halves of a register; nibbles by one three-input logic instruction, where
// those of a byte's upper half make 1024 + 16 n and are not shifted down: their factor of 16 is
// taken into the other operand of the product (or out of its result), exactly.
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

// Where the codes of token t of a block are that belong to chunk k's 32-bit word `word` (8 or 4 columns): K's
// are the word; V's are its four bytes, in pieces of 2 bytes (4 bits) or of 1, each as far from the next as two pieces.
__device__ __forceinline__ int q_k_at(int chunks, int t, int k, int word) {
  return ((t >> 3) * chunks + k) * 128 + (t & 7) * 16 + word * 4;
}
__device__ __forceinline__ int q_v_at(int bits, int chunks, int t, int k, int word) {
  return ((t >> 3) * chunks + k) * 128 + (t & 7) / 2 * 32 + word * 8 + (t & 1) * (bits == 4 ? 2 : 1);
}
// A token's word of V codes, and its place in memory
template <int BITS>
__device__ __forceinline__ void q_v_store(uint8_t* at, uint32_t w) {
  if constexpr (BITS == 4) {
    reinterpret_cast<uint16_t*>(at)[0] = (uint16_t)w;
    reinterpret_cast<uint16_t*>(at)[2] = (uint16_t)(w >> 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) at[2 * i] = (uint8_t)(w >> (8 * i));
  }
}
// (8 bits: both tokens' codes in two aligned words)
__device__ __forceinline__ uint32_t q_v_load8(const uint8_t* at) {
  const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<uintptr_t>(at) & ~(uintptr_t)7);
  return __byte_perm(v.x, v.y, reinterpret_cast<uintptr_t>(at) & 1 ? 0x7531 : 0x6420);
}

__device__ __forceinline__ float q_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float q_offset(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Two codes of a word as 1024 + code, and 1024 + 16 code for nibbles 1 and 3 of a half. 4 bits: nibbles
// R and R + 4 (R = 0 .. 3). 8 bits: bytes 2 R and 2 R + 1 (R = 0, 1). `raised`: Q_RAISED, from where the
// compiler does not see its value: it would make two instructions of an and with one constant and an or with another.
constexpr uint32_t Q_RAISED = 0x64006400u;
template <int BITS, int R>
__device__ __forceinline__ uint32_t q_raise(uint32_t w, uint32_t raised) {
  if constexpr (BITS == 8) return __byte_perm(w, raised, R == 0 ? 0x5150 : 0x5352);
  else return ((R < 2 ? w : w >> 8) & (R % 2 ? 0x00f000f0u : 0x000f000fu)) | raised;
}
// The same with all nibbles as 1024 + 16 n, so that one factor serves all (two shifts more).
template <int BITS, int R>
__device__ __forceinline__ uint32_t q_raise16(uint32_t w, uint32_t raised) {
  if constexpr (BITS == 8) return q_raise<8, R>(w, raised);
  else return ((R == 0 ? w << 4 : R == 1 ? w : w >> (4 * R - 4)) & 0x00f000f0u) | raised;
}
// Two codes of a word as fp16 numbers below the normal ones, 2^-24 times the code (times 16 for nibbles 1 and 3 of a
// half): nothing to set and no constant to take off. (fp16 products are exact for these too.)
template <int BITS, int R>
__device__ __forceinline__ uint32_t q_small(uint32_t w) {
  if constexpr (BITS == 8) return __byte_perm(w, 0u, R == 0 ? 0x4140 : 0x4342);
  else return (R < 2 ? w : w >> 8) & (R % 2 ? 0x00f000f0u : 0x000f000fu);
}
// A scale times 2^24 (one multiply-add; of zero it is 2^-103, whose codes are all zero, and of NaN a number, whose offset
// is NaN)
__device__ __forceinline__ float q_scale24(uint32_t p) { return __uint_as_float(p * 65536u + (24u << 23)); }
template <int BITS>
__host__ __device__ constexpr float q_factor(int r) { return BITS == 4 && r % 2 ? 16.f : 1.f; }

// Their constants taken off, 8 or 128 (times the factor) with them: with the codes' mean near zero their
// sums lose nothing to a constant that is many times as large as what is summed up. Exact.
template <int BITS, int R>
__device__ __forceinline__ uint32_t q_centred(uint32_t raised) {
  constexpr uint32_t MINUS = BITS == 8 ? 0xe480e480u /* 1152 */ : R % 2 ? 0xe480e480u : 0xe408e408u /* 1032 */;
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(raised), "r"(MINUS));
  return d;
}

__device__ __forceinline__ uint32_t q_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t q_mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t q_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// From here on a score (log2) is rounded before its row's reference m, one such score, is taken off. Below it the two are one
// fused operation, in which the largest score keeps what m was rounded by, half an ulp of m: 2^5 of 2^30, by which its
// probability would be 2^32, or 2^-32 and the row's sum 0.
constexpr float Q_LARGE = 0x1p20f;
__device__ __forceinline__ float q_pow2(int e) { return __int_as_float((e + 127) << 23); }      // -126 <= e <= 127
__device__ __forceinline__ int q_exponent(float x) { return (__float_as_int(x) >> 23) - 127; }  // of x > 0

fa_status launch_qappend(const void* q, const void* k, const void* v, void* qo, const int* cu, const int* slots,
                         const fakv_rope* r, const QCache& c, const fakv_tokens& p, cudaStream_t s);
fa_status launch_qread(void* K, void* V, const int* cu, const int* slots, const int* first, const QCache& c,
                       const fakv_tokens& p, cudaStream_t s);
fa_status launch_qattend_rows(const void* q, void* O, float* LSE, const int* cu, const int* slots, const QCache& c,
                              const fakv_tokens& p, cudaStream_t s);
fa_status launch_qattend_tiles(const void* q, void* O, float* LSE, const int* cu, const int* slots, const QCache& c,
                               const fakv_tokens& p, cudaStream_t s);

}  // namespace kv
}  // namespace fa
