// kv_tiles.cu -- attention over a bf16 paged cache, or one in 4 or 8 bits, for many rows per sequence (chunks of
// a prompt): TMA from the pages (codes: warps that make fp16 of them), tcgen05, TMEM.
//
// Many rows per key make the work 4 D flops per (row, key) on the tensor cores. An item is
// two 128-row tiles of one sequence and kv head: the rows of a tile are tpt tokens x the
// rep query heads that read the kv head (tpt = 128 / rep), so K and V are fetched once for
// all of them whatever rep is. A CTA (one per SM) walks its part of the work line
// (kv_sched.cuh) in units of 128 keys, copied page by page: a tile of 128 keys is the
// boxes of 128 / page_size pages (each lane of a producer warp issues one), laid one after
// another in shared memory as if the keys were contiguous.
//
// Roles, rings and hand-offs are those of fa_fwd_kernel, the items being the segments of the
// part:
//   warps 0 - 7   softmax, four per tile: thread = row = TMEM lane
//   warp 8        MMA issuer: S_q = Q_q K^T, O_q += P_q V, tiles alternating
//   warp 9, 10    producers: Q and K, V (and the epilogue's stages)
//   warp 11       relay of landed copies to the issuer; it also zeroes V's rows past a
//                 sequence's end, whose memory may hold anything (0 x NaN)
// A wait that runs out raises the CTA's abort flag. Named barriers have no limit, so their
// rounds are all joined nevertheless: the relay and the issuer go on with whatever the stages
// hold, and the softmax warps wait for the issuer whatever the flag says (a warp that gave up
// between two rounds could complete a neighbour's); producers and epilogues, whose waits are
// all on mbarriers, stop. tests/test_kv_tiles_sync_model.py replays all of it.
// P is one bf16 term where O is bf16: its rounding, at most 2^-8 of a probability and
// random in sign, adds to O about what O's own rounding does (2048 tokens over 16384: O is
// 2.4e-3 of its size from the 64-bit values, 1.7e-3 of that its own rounding), and a second
// term would take 560 to 600 us where one takes 341. An fp32 O has no such rounding to hide
// behind: with one term it would be 1.7e-3 off too. There P is two terms (2^-16), the second
// in the half of S's TMEM columns that the first leaves free: 3e-5 off (8192 tokens of a
// prompt: 650 to 690 us against 385). It is not the tensor pipe that fills then (60 %) but
// the softmax warps' extra terms and TMEM stores.
//
// Measured: 2048 tokens over 16384 (32 query heads on 8 of 128) 305 to 317 us with the join, 1660
// TFLOP/s, 0.86 of the measured peak (333 to 337 with the MMAs issued by lane 0 and each descriptor put together anew; the
// figures that follow, and those of two terms above, are of that form); 8192 tokens of a prompt 385 us, 0.75. A unit of 128
// keys takes a CTA 2720 clocks, of which its MMAs fill 2240: a tile's softmax (1130 clocks: 62 to
// load the scores, 320 for the maximum, 690 for the exponentials) and the hand-offs on both
// sides of it are longer than the other tile's MMAs. Tried, and slower: two threads to a row
// (640 threads leave 96 registers each: it spilled, 633 us), and P handed over in two halves
// (2820 clocks). An item costs 4 us besides its units (epilogue, first scores), which the
// schedule counts as three units; the start of the kernel 8 us.
//
// Codes of 4 or 8 bits (640 threads). Four roles are different:
//   warps 12 - 19 codes: each writes an eighth of K's and of V's tile as fp16, in turn, where bf16's copies would have
//                 laid them (the comment at their branch has the numbers' form)
//   warp 9        producer of q alone, which qattend_q_kernel has made fp16 before; warp 10 has nothing to do
//   warps 0 - 7   the softmax takes 64 keys at a time, its 128 registers having no room for more; P is fp16
// Three programs at once run an SM's warps out of instruction memory, so the loops over octets and over 64 keys are not
// unrolled, and what keys of very different sizes need (powers of two of their own) goes through tensor memory in small loops
// behind one vote (2048 tokens over 16384 in 4 bits: 1097 us with all unrolled, 487 now; 514 with a branch on what the code warps had written).
// That is 0.55 of the tensor peak at 2.4 us to a unit, of which its MMAs, K's offsets among them, fill 1.45. In the form of 475
// us, without powers of two by key and row: without turning codes into numbers 424, with half of a softmax 380, without either
// 338. Eight bits: K's two planes double the first product
// and leave room for one stage of K, so that a unit is its codes, then both tiles' products, in turn (3.9 us; six
// chunks of up to 500 tokens 89 us; 91 with the factors formed after the wait for the stage). Tried, and slower or the same
// (the codes' form of 479 us): 640 threads split 136/48/80 and 128/64/80 registers, three octets of
// 8-bit codes ahead, products over the columns that there are (96 of 128 by a branch in the issuer: 577 us for 479; by a kernel of its own 86 for
// 89, too little for two more), four warps for K
// and four for V (511; K's are then what all wait for), codes in registers a tile ahead. tests/test_kvq_tiles_sync_model.py
// replays these hand-offs.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include "kv_quant.cuh"
#include "kv_sched.cuh"

namespace fa {
namespace kv {

static __device__ unsigned int g_kv_status = 0;

namespace {
using namespace ptx;

struct TilesArgs {
  fakv_cache c;
  QCache qc;         // codes
  uint32_t raised;   // Q_RAISED
  const float* qf;   // codes: what makes logits (log2) of a row's scores, [T][H]
  void* O;
  float* LSE;
  const int* cu;
  const int* slots;
  int B, T, H, shift;
  int RT, tpt;      // rows and tokens of a tile
  int box, boxes;   // keys of a page box, boxes of a key tile
  Geo g;
  float sl2;
  int out_bf16;
  Partials part;
  unsigned long long limit_ns;
};

template <int D_, int BITS>  // BITS: of the cache's codes; 0: bf16 pages
struct TilesCfg {
  static constexpr int D = D_;
  static constexpr int NQ = 2;
  static constexpr uint32_t FMT = BITS ? FMT_F16 : FMT_BF16;
  static constexpr bool CODES = BITS != 0;
  static constexpr int NCB = D / 64;                      // 64-column blocks
  static constexpr uint32_t CB_BYTES = 128u * 128u;       // one block of a 128-row tile
  static constexpr uint32_t TILE_BYTES = NCB * CB_BYTES;
  // codes of 8 bits: K in two planes (see the code warps), of a stage
  static constexpr int PLANES = BITS == 8 ? 2 : 1;
  static constexpr int KST = BITS == 8 ? (D == 128 ? 1 : 2) : D == 128 ? 2 : 3;
  static constexpr uint32_t K_STAGE = PLANES * TILE_BYTES;
  static constexpr int VST = BITS ? 2 : 3;
  static constexpr uint32_t EPI_BOX = 32u * 128u;         // a warp's staging: 32 rows x 128 bytes
  static constexpr uint32_t V_STAGE = std::max(TILE_BYTES, 4 * NQ * EPI_BOX);
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t K_OFF = Q_OFF + NQ * TILE_BYTES;
  static constexpr uint32_t V_OFF = K_OFF + KST * K_STAGE;
  static constexpr uint32_t OCTET = D * BITS;              // bytes of eight keys' codes
  static constexpr int AHEAD = PLANES == 2 ? 2 : 4;        // octets on their way to a code warp (four to a tile)
  static constexpr uint32_t RING = AHEAD * OCTET;
  static constexpr uint32_t CODES_OFF = V_OFF + VST * V_STAGE;
  // codes: eight columns more of Q and K, for the offsets (and eight of zeros to make up the product's sixteen)
  static constexpr uint32_t MORE = 128u * 16u;
  static constexpr uint32_t QMORE_OFF = CODES_OFF + 8 * RING, KMORE_OFF = QMORE_OFF + NQ * MORE, ZERO_OFF = KMORE_OFF + KST * MORE;
  static constexpr uint32_t SMEM = (BITS ? ZERO_OFF + MORE : CODES_OFF) + 1024;
  static constexpr int SOFTMAX_WARPS = 8, MMA_WARP = 8, KQ_WARP = 9, V_WARP = 10, RELAY_WARP = 11;
  static constexpr uint32_t RELAY_BAR = 3;  // named barrier (1 + q: P_q written)
  static constexpr int CODE_WARP = 12;  // codes: eight warps, an eighth of each tile
  static constexpr int THREADS = BITS ? 640 : 384;
  static constexpr uint32_t REGS_SOFTMAX = BITS ? 128 : 216, REGS_CONTROL = BITS ? 48 : 64, REGS_CODES = 88;
  static_assert(2 * 128 * REGS_SOFTMAX + 128 * REGS_CONTROL + (BITS ? 256 * REGS_CODES : 0) <= (BITS ? 640 * 96 : 384 * 168),
                "register split exceeds the launch allocation");
  static constexpr uint32_t FILLERS = BITS ? 8 : 1;  // arrivals at a landed tile's barrier, and at a grant
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t s_col(int q) { return 128u * q; }
  __host__ __device__ static constexpr uint32_t o_col(int q) { return 256u + (uint32_t)D * q; }
  static_assert(SMEM <= 227u * 1024u, "shared memory budget");
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One lane of a converged warp, the same one each time. (The MMAs' operands are then known to be the same for all
// lanes that get there: chunks in 4 bits 489 us with lane 0 by comparison, 480 with this; in 8 bits 95 and 92.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p)::"memory");
  return p != 0;
}
template <class C>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t sq, uint32_t sk, uint32_t q_more, uint32_t k_more, uint32_t zero) {
  constexpr uint32_t id = make_idesc(128, 128, C::FMT, C::FMT, false, false);
  // (rows of 16 bytes, without a swizzle: eight rows 128 bytes on, the next eight columns -- zeros -- where `zero` is)
  if (C::CODES) mma_f16_ss(d_tmem, make_sdesc(q_more, zero - q_more, 128, 0), make_sdesc(k_more, zero - k_more, 128, 0), id, 0);
  const uint64_t dq = make_sdesc(sq, 16, SW128_ATOM), dk = make_sdesc(sk, 16, SW128_ATOM);
#pragma unroll
  for (int plane = 0; plane < C::PLANES; ++plane)
#pragma unroll
    for (int kk = 0; kk < C::D / 16; ++kk) {  // (no address carries past its field)
      const uint32_t off = (kk / 4) * C::CB_BYTES + (kk % 4) * 32;
      mma_f16_ss(d_tmem, dq + off / 16, dk + (plane * C::TILE_BYTES + off) / 16, id, kk > 0 || C::CODES);
    }
}
template <class C, int TERMS>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t sv, bool accumulate) {
  constexpr uint32_t id = make_idesc(128, C::D, C::FMT, C::FMT, false, true);
  const uint64_t dv = make_sdesc(sv, C::CB_BYTES, SW128_ATOM);
#pragma unroll
  for (int term = TERMS - 1; term >= 0; --term)
#pragma unroll
    for (int kk = 0; kk < BLOCK_N / 16; ++kk)
      mma_f16_ts(o_tmem, p_tmem + term * 64 + kk * 8, dv + kk * 128, id,
                 (accumulate || kk > 0 || term < TERMS - 1) ? 1u : 0u);
}

// 32 accumulator rows of a warp, times mul, to row_ptr(r) (null: not written), staged in a
// 32 x 128-byte box of shared memory so that stores are whole 128-byte lines.
template <int D, bool BF, typename RowPtr>
__device__ __forceinline__ void store_rows(uint32_t t_addr, bool have, float mul, uint32_t stage, int cols,
                                           RowPtr row_ptr) {
  constexpr int COLS = BF ? 64 : 32;
  const uint32_t lane = lane_id(), sw = lane & 7u;
  const uint32_t row = stage + lane * 128u;
  const int rr = (int)(lane >> 3), ch = (int)(lane & 7u);
  char* to[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) to[i] = row_ptr(rr + 4 * i);
#pragma unroll 1
  for (int b = 0; b * COLS < cols; ++b) {
    if constexpr (BF) {
      uint32_t r0[32], r1[32];
      if (have) {
        tmem_ld32x2(t_addr + b * 64, t_addr + b * 64 + 32, r0, r1);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) r0[k] = r1[k] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = (c % 4) * 8 + 2 * e;
          w[e] = pack_bf2(__uint_as_float(c < 4 ? r0[k] : r1[k]) * mul, __uint_as_float(c < 4 ? r0[k + 1] : r1[k + 1]) * mul);
        }
        st_shared_v4(row + ((c ^ sw) << 4), w[0], w[1], w[2], w[3]);
      }
    } else {
      uint32_t r[32];
      if (have) {
        tmem_ld32(t_addr + b * 32, r);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) r[k] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_v4(row + ((c ^ sw) << 4), __float_as_uint(__uint_as_float(r[4 * c]) * mul),
                     __float_as_uint(__uint_as_float(r[4 * c + 1]) * mul),
                     __float_as_uint(__uint_as_float(r[4 * c + 2]) * mul),
                     __float_as_uint(__uint_as_float(r[4 * c + 3]) * mul));
    }
    __syncwarp();
    const int col = b * COLS + ch * (BF ? 8 : 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rl = rr + 4 * i;
      const float4 v = ld_shared_v4(stage + (uint32_t)rl * 128u + (((uint32_t)ch ^ ((uint32_t)rl & 7u)) << 4));
      if (to[i] && col < cols) *reinterpret_cast<float4*>(to[i] + col * (BF ? 2 : 4)) = v;
    }
    __syncwarp();
  }
  fence_async_shared();  // before the copy engine writes the stage again
}

// ---- tiles of codes
// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void cp_piece(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
constexpr int TILE_INFO = 8;  // tiles whose powers of two are kept: K's codes are at most five tiles ahead of the softmax
constexpr int SPREAD = 3;     // log2 of how far below the largest of 32 keys a key may be and share its powers of two
constexpr float OWN = 1024.f; // added to V's exponent of 32 keys that have their own

// q as fp16, each row times a power of two that brings its largest value to 2^14 (exactly, but for what is 2^-28 of
// that), and what undoes it, times the softmax scale; `pairs`: each eight columns in the order 0 4 1 5 2 6 3 7, which is
// that of K's 4-bit codes. Beside it eight columns more, for K's offsets: of each group the sum S of q, times 2^-8, as
// two fp16 terms, high, low and high again (for the offset's high, high and low term). Sixteen lanes to a row. A row with
// NaN or infinity becomes NaN.
constexpr int QROWS_THREADS = 256;
constexpr float Q_SUM = 0x1p-8f;
__global__ void __launch_bounds__(QROWS_THREADS) qattend_q_kernel(const __nv_bfloat16* q, long long q_token, long long q_head,
                                                                  int rows, Div heads, int D, int groups, float sl2, bool pairs,
                                                                  uint16_t* out, uint4* more, float* factor) {
  grid_launch_dependents();
  const int lane = threadIdx.x & 15, row = blockIdx.x * (QROWS_THREADS / 16) + threadIdx.x / 16;
  const int token = heads.of(min(row, rows - 1)), col = lane * 8;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (row < rows && col < D)
    v = *reinterpret_cast<const uint4*>(q + token * q_token + (row - token * heads.d) * q_head + col);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8], top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(x[i]));
    fine = fine && fabsf(x[i]) < INFINITY;
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    fine = __shfl_xor_sync(0xffffffffu, (int)fine, d) && fine;
  }
  const int e = min(max(q_exponent(top), -100), 127);
  const float by = fine ? q_pow2(14 - e) : __int_as_float(0x7fffffff);
  uint32_t y[4];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = q_half2((pairs ? x[i] : x[2 * i]) * by, (pairs ? x[i + 4] : x[2 * i + 1]) * by);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
    sum += f.x + f.y;
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  float other = __shfl_xor_sync(0xffffffffu, sum, 8);  // (of the second group, in the first lane)
  if (groups == 1) {
    sum += other;
    other = 0.f;
  }
  if (row >= rows) return;
  if (col < D) *reinterpret_cast<uint4*>(out + (size_t)row * D + col) = make_uint4(y[0], y[1], y[2], y[3]);
  if (lane == 0) {
    const uint32_t h = q_half2(sum * Q_SUM, other * Q_SUM);  // (low half: first group)
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const uint32_t l = q_half2(sum * Q_SUM - f.x, other * Q_SUM - f.y);
    // h0 l0 | h0 h1 | l1 h1 | 0 0
    more[row] = make_uint4(__byte_perm(h, l, 0x5410), h, __byte_perm(l, h, 0x7632), 0u);
    factor[row] = sl2 * q_pow2(e - 14);
  }
}

template <int D, int TERMS, int BITS>
__global__ void __launch_bounds__(TilesCfg<D, BITS>::THREADS, 1)
    attend_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TilesArgs a) {
  // (codes: K and V have no map; tmK is that of q's columns more)
  using C = TilesCfg<D, BITS>;
  constexpr int NQ = C::NQ, KST = C::KST, VST = C::VST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_q[NQ], bar_qfree[NQ], bar_kfull[KST], bar_kempty[KST], bar_vfull[VST],
      bar_vempty[VST], bar_grant[NQ], bar_s[NQ], bar_o[NQ], bar_join, bar_drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, stuck_sh;
  // codes: of each quarter of a tile, K's power of two and V's exponent, or 1 and V's exponent + OWN, and of each key of that
  // quarter K's power of two (the high half is its bits) and V's (the low half)
  __shared__ float2 info_sh[BITS ? TILE_INFO : 1][4];
  __shared__ uint32_t keys_sh[BITS ? TILE_INFO : 1][BITS ? 128 : 1];
  __shared__ PlanShared<C::THREADS, 1> plan;
  grid_launch_dependents();
  const int warp = warp_id(), lane = lane_id();
  volatile int* abort_flag = &abort_sh;
  volatile int* stuck_flag = &stuck_sh;
  if (threadIdx.x == 0) {
    for (int q = 0; q < NQ; ++q) {
      mbar_init(&bar_q[q], 1);
      mbar_init(&bar_qfree[q], 1);
      mbar_init(&bar_s[q], 1);
      mbar_init(&bar_o[q], 1);
      mbar_init(&bar_grant[q], C::FILLERS);
    }
    for (int s = 0; s < KST; ++s) { mbar_init(&bar_kfull[s], C::FILLERS); mbar_init(&bar_kempty[s], 1); }
    for (int s = 0; s < VST; ++s) { mbar_init(&bar_vfull[s], C::FILLERS); mbar_init(&bar_vempty[s], 1); }
    mbar_init(&bar_join, C::SOFTMAX_WARPS);
    mbar_init(&bar_drain, 1);
    abort_sh = stuck_sh = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2) a.part.left[2 * blockIdx.x + threadIdx.x].flags = 0;
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish();
  }
  Seq seq;
  const Part part = find_part<C::THREADS, 1>(a.g, a.c, a.cu, a.slots, a.B, a.T, reinterpret_cast<int*>(smem), plan, seq);
  if constexpr (BITS != 0) {
    if (threadIdx.x < C::MORE / 16) st_shared_v4(smem_u32(smem) + C::ZERO_OFF + threadIdx.x * 16, 0, 0, 0, 0);
    grid_dependency_wait();  // (q as fp16)
  }
  // (the plan's scratch lies in the tiles: its generic accesses before the copies' writes)
  fence_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const uint32_t sbase = smem_u32(smem);
  auto sQ = [&](int q) { return sbase + C::Q_OFF + q * C::TILE_BYTES; };
  auto sK = [&](int st) { return sbase + C::K_OFF + st * C::K_STAGE; };
  auto sQmore = [&](int q) { return sbase + C::QMORE_OFF + q * C::MORE; };
  auto sKmore = [&](int st) { return sbase + C::KMORE_OFF + st * C::MORE; };
  auto sV = [&](int st) { return sbase + C::V_OFF + st * C::V_STAGE; };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, abort_flag, &g_kv_status, DEV_TIMEOUT, a.limit_ns);
  };
  // of a producer: a stage given back after an abort is not filled again
  auto wait_free = [&](uint64_t* bar, uint32_t parity) { return wait(bar, parity) && !*abort_flag; };
  // for the issuer, who goes on after an abort (all other waits have run out by twice their limit)
  auto wait_issuer = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, stuck_flag, &g_kv_status, DEV_TIMEOUT, 2 * a.limit_ns);
  };
  auto drain = [&](uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < a.limit_ns) {}
  };
  Walk walk(part, seq);
  Seg seg;
  auto next = [&]() { return walk.next(a.g, a.c, a.cu, a.slots, a.T, seg); };

  // A producer lane's box of key tile kt: its page (num_pages, past the tensor, where no
  // row sees its keys or the table names none: zeros are filled in)
  const int my_box = lane % a.boxes, my_cb = lane / a.boxes;
  auto page_for = [&](int kt) {
    const int j = kt * BLOCK_N + my_box * a.box;
    int p = a.c.num_pages;
    if (j < seg.x.hi && j + a.box > seg.x.lo) {
      p = a.c.table[(long long)seg.s.slot * a.c.table_stride + (j >> a.shift)];
      if ((unsigned)p >= (unsigned)a.c.num_pages) {
        raise(a.c.status, FAKV_BAD_PAGE);
        p = a.c.num_pages;
      }
    }
    return p;
  };
  auto load_tile = [&](uint32_t dst, const CUtensorMap* map, uint64_t* bar, int kt, int page) {
    if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE_BYTES);
    __syncwarp();
    if (my_cb < C::NCB)
      tma_load_4d(dst + my_cb * C::CB_BYTES + my_box * a.box * 128, map, bar, my_cb * 64,
                  (kt * BLOCK_N + my_box * a.box) & (a.c.page_size - 1), seg.head, page);
    __syncwarp();
  };

  if (BITS && warp >= C::CODE_WARP) {
    // ------------------------------------------------------------ codes of K, of V
    // Each of four warps writes 32 keys of every tile, as the copies of bf16 pages would have laid them down, in fp16:
    // times a power of two that keeps the largest of the 32 keys' values just below 2^4 (K: undone in the scores) or
    // 2^7 (V: undone in the probabilities). V is x s + z', rounded to 2^-11 of it. A score's error moves a probability by
    // its factor, so K is not rounded: x s of a nibble x in -8 .. 7 has the eleven bits of fp16 (of a byte it is two such
    // terms, 16 (h - 8) s and (l - 8) s, in two planes), and z' (two terms) is multiplied with the row's sum of q in one
    // step of the product more. (K as x s + z' in one term had LSEs 8e-6 off, and 3e-5 where few keys were seen.) Where one
    // of the 32 keys is 2^SPREAD below the largest, or K's scale too small to be exact, each key has powers of two of its
    // own, which the softmax undoes key by key: no key costs another's bits, least of all one that a row does not see. The
    // codes are on their way while those before are turned into numbers. Keys that no row sees, and those of a missing page,
    // are zeros; a key whose scale is NaN, in K or in V, is NaN in K and zeros in V, so that rows that see it become NaN
    // and the tile's others do not.
    regs_decrease<C::REGS_CODES>();
    if constexpr (BITS != 0) {
        constexpr int CH = D * BITS / 128, PIECES = CH >= 4 ? CH / 4 : 1;  // chunks of a key; a lane's pieces of an octet
        constexpr int NG = D / 64;
        constexpr float V_CENTRE = BITS == 4 ? 8.f : 128.f, K_CENTRE = BITS == 4 ? 8.f : 136.f, STEPS = BITS == 4 ? 15.f : 255.f;
        const int quarter = (warp - C::CODE_WARP) >> 1, half = warp & 1;  // of the tile; of the quarter
        const int chunks = a.qc.chunks, ng = a.qc.groups;
        const uint32_t ring = sbase + C::CODES_OFF + (warp - C::CODE_WARP) * C::RING;
        // the lane's piece, 16 bytes of an octet's 128 a chunk. K: chunk chunk0 of token lane % 8. V: half a pair's
        // chunk, both tokens'.
        const int chunk0 = lane >> 3, side = (lane >> 2) & 1;
        auto piece_at = [&](bool is_v) { return chunk0 * 128 + (is_v ? (lane & 3) * 32 + side * 16 : (lane & 7) * 16); };
        auto octet_page = [&](int kt) {  // of octet lane / 8 of the warp's quarter: -1: unseen or missing
          const int j = kt * BLOCK_N + quarter * 32 + (lane & ~7);
          if (j >= seg.x.hi || j + 8 <= seg.x.lo) return -1;
          const int p = a.c.table[(long long)seg.s.slot * a.c.table_stride + (j >> a.shift)];
          if ((unsigned)p < (unsigned)a.c.num_pages) return p;
          raise(a.c.status, FAKV_BAD_PAGE);
          return -1;
        };
        // params of key `lane` of the quarter, K's and V's
        struct Params {
          uint32_t k[NG], v[NG];
        };
        auto ask_params = [&](Params& b, int kt, int page) {
          const int key = kt * BLOCK_N + quarter * 32 + lane;
          const long long off = page * a.qc.page + seg.head * a.qc.head + a.qc.params + (key & (a.c.page_size - 1)) * ng * 4;
          const bool in = page >= 0 && key >= seg.x.lo && key < seg.x.hi;
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            const int w = NG > 1 && ng > 1 ? j * 4 : 0;
            b.v[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(a.qc.V + off + w)) : 0u;
            b.k[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(a.qc.K + off + w)) : 0u;
          }
        };
        // a warp's octets of a tile, in turn: two of K, two of V (each piece read by the lane that asked for it)
        auto ask = [&](int kt, int page, int turn) {
          const int octet = 2 * half + (turn & 1);
          const uint8_t* const base = turn < 2 ? a.qc.K : a.qc.V;
          const int at = piece_at(turn >= 2);
          const int p = __shfl_sync(0xffffffffu, page, octet * 8);
          const int t = (kt * BLOCK_N + quarter * 32 + octet * 8) & (a.c.page_size - 1);
          const uint8_t* const from = base + max(p, 0) * a.qc.page + seg.head * a.qc.head + t * chunks * 16;
#pragma unroll
          for (int z = 0; z < PIECES; ++z) {
            const bool take = p >= 0 && chunk0 + 4 * z < chunks;
            if (chunk0 + 4 * z < CH) cp_piece(ring + turn % C::AHEAD * C::OCTET + at + z * 512, take ? from + at + z * 512 : base, take);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // scale (low) and z' (high) of key `lane`, as fp16 times the quarter's power of two
        struct Factors {
          uint32_t f[NG];
          float z[2];  // K: z' in fp32, of the first and of the second group
        };
        auto nan = [](const uint32_t (&p)[NG]) {
          bool bad = false;
#pragma unroll
          for (int j = 0; j < NG; ++j) bad |= (p[j] & 0x7fffu) > 0x7f80u;
          return bad;
        };
        auto exponent_of = [&](const uint32_t (&p)[NG]) {  // of the largest value that the key can hold
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < NG; ++j)
            top = fmaxf(top, fmaxf(fabsf(q_offset(p[j])), fabsf(fmaf(q_scale(p[j]), STEPS, q_offset(p[j])))));
          if (nan(p)) top = 0.f;
          return min(max(q_exponent(top), -100), 126);
        };
        // the exponents that key `lane` of the quarter is written with: the largest of the 32, or its own
        struct Exponents {
          int k, v;
        };
        auto exponents = [&](const Params& b, int kt, int g) {
          const int own_k = exponent_of(b.k), own_v = exponent_of(b.v), key = kt * BLOCK_N + quarter * 32 + lane;
          Exponents e = {__reduce_max_sync(0xffffffffu, own_k), __reduce_max_sync(0xffffffffu, own_v)};
          const float by = q_pow2(3 - e.k);
          // (a K of zeros is as good with any exponent; a V of zeros that some row sees is not to stand for a larger one. A key
          // that is NaN has no say: rows that see it are NaN)
          bool apart = (own_k > -100 && own_k < e.k - SPREAD) ||
                       (own_v < e.v - SPREAD && key >= seg.x.lo && key < seg.x.hi && !nan(b.k) && !nan(b.v));
#pragma unroll
          for (int j = 0; j < NG; ++j) apart |= q_scale(b.k[j]) > 0.f && q_scale(b.k[j]) * by < 0x1p-17f;
          const float v_top = (float)(e.v - 6);
          if (__any_sync(0xffffffffu, apart)) {
            e = {own_k, own_v};
            if (half == 0) keys_sh[g % TILE_INFO][quarter * 32 + lane] = (uint32_t)(own_k + 124) << 23 | (uint32_t)(own_v + 121) << 7;
            if (half == 0 && lane == 0) info_sh[g % TILE_INFO][quarter] = make_float2(1.f, v_top + OWN);
          } else if (half == 0 && lane == 0) {
            info_sh[g % TILE_INFO][quarter] = make_float2(q_pow2(e.k - 3), v_top);
          }
          return e;
        };
        auto factors = [&](auto is_v, const Params& b, const Exponents& exps) {
          constexpr bool IS_V = decltype(is_v)::value;
          const int e = IS_V ? exps.v - 6 : exps.k - 3;
          const float by = q_pow2(-e);
          const bool bad = nan(b.v) || (!IS_V && nan(b.k));
          Factors f;
          f.z[0] = f.z[1] = 0.f;
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            const uint32_t p = IS_V ? b.v[j] : b.k[j];
            const float s = q_scale(p), z = fmaf(s, IS_V ? V_CENTRE : K_CENTRE, q_offset(p)) * by;
            f.f[j] = bad ? (IS_V ? 0u : 0x7fff7fffu) : q_half2(s * by, z);
            if constexpr (!IS_V) f.z[j] = bad || (j > 0 && ng == 1) ? 0.f : z;
          }
          return f;
        };
        auto write = [&](auto is_v, const Factors& f, uint32_t tile, int turn) {
            constexpr bool IS_V = decltype(is_v)::value;
            const int octet = 2 * half + (turn & 1), token = IS_V ? 2 * (lane & 3) : lane & 7, at = piece_at(IS_V);
            const int r = quarter * 32 + octet * 8 + token;  // row of the tile
            uint32_t sz[NG][IS_V ? 2 : 1];
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
              for (int e = 0; e < (IS_V ? 2 : 1); ++e) sz[j][e] = __shfl_sync(0xffffffffu, f.f[j], octet * 8 + token + e);
#pragma unroll
            for (int z = 0; z < PIECES; ++z) {
              const int col = (chunk0 + 4 * z) * (128 / BITS);
              if (col >= D) continue;
              // 16-byte piece c of row r + e
              auto put = [&](int e, int c, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t plane = 0) {
                st_shared_v4(tile + plane + (c >> 3) * C::CB_BYTES + (r + e) * 128 + (((c & 7) ^ ((r + e) & 7)) << 4), x0, x1, x2, x3);
              };
              const bool upper = NG > 1 && col >= 64;
              const uint32_t p0 = upper ? sz[NG - 1][0] : sz[0][0], p1 = IS_V ? (upper ? sz[NG - 1][IS_V] : sz[0][IS_V]) : p0;
              const uint32_t s = __byte_perm(p0, p1, 0x5410), zz = __byte_perm(p0, p1, 0x7632);
              const float4 piece = ld_shared_v4(ring + turn % C::AHEAD * C::OCTET + at + z * 512);
              const uint32_t words[4] = {__float_as_uint(piece.x), __float_as_uint(piece.y), __float_as_uint(piece.z), __float_as_uint(piece.w)};
              if constexpr (BITS == 4) {
                const uint32_t s16 = q_mul2(s, 0x2c002c00u);  // s / 16
                // the four pairs of a word: K: columns n and n + 4; V: column n of both tokens
                auto number = [&](uint32_t x, uint32_t by) { return IS_V ? q_fma2(x, by, zz) : q_mul2(x, by); };
                auto pairs = [&](uint32_t w, uint32_t (&x)[4]) {
                  x[0] = number(q_centred<4, 0>(q_raise<4, 0>(w, a.raised)), s);
                  x[1] = number(q_centred<4, 1>(q_raise<4, 1>(w, a.raised)), s16);
                  x[2] = number(q_centred<4, 2>(q_raise<4, 2>(w, a.raised)), s);
                  x[3] = number(q_centred<4, 3>(q_raise<4, 3>(w, a.raised)), s16);
                };
                if constexpr (!IS_V) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    uint32_t x[4];
                    pairs(words[i], x);
                    put(0, col / 8 + i, x[0], x[1], x[2], x[3]);  // (columns 0 4 1 5 2 6 3 7, as q's are laid)
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    // (the two sides' lanes take their words in turn, so that eight lanes' pieces lie in different banks)
                    const int k = i ^ side;
                    uint32_t x[4], y[4];
                    pairs(k ? words[2] : words[0], x);
                    pairs(k ? words[3] : words[1], y);
                    put(0, col / 8 + side * 2 + k, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                        __byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410));
                    put(1, col / 8 + side * 2 + k, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632),
                        __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
                  }
                }
              } else {
                uint32_t x[4][2];  // of each word, K: columns 0, 1 and 2, 3; V: column 0 and column 1 of both tokens
                if constexpr (!IS_V) {
#pragma unroll
                  for (int plane = 0; plane < 2; ++plane) {  // 16 h, then l
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const uint32_t r0 = q_raise<8, 0>(words[k], a.raised), r1 = q_raise<8, 1>(words[k], a.raised);
                      x[k][0] = q_mul2(plane ? q_centred<4, 0>(r0 & 0xff0fff0fu) : q_centred<4, 1>(r0 & 0xfff0fff0u), s);
                      x[k][1] = q_mul2(plane ? q_centred<4, 0>(r1 & 0xff0fff0fu) : q_centred<4, 1>(r1 & 0xfff0fff0u), s);
                    }
                    put(0, col / 8, x[0][0], x[0][1], x[1][0], x[1][1], plane * C::TILE_BYTES);
                    put(0, col / 8 + 1, x[2][0], x[2][1], x[3][0], x[3][1], plane * C::TILE_BYTES);
                  }
                } else {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    x[k][0] = q_fma2(q_centred<8, 0>(q_raise<8, 0>(words[k], a.raised)), s, zz);
                    x[k][1] = q_fma2(q_centred<8, 1>(q_raise<8, 1>(words[k], a.raised)), s, zz);
                  }
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t sel = e ? 0x7632 : 0x5410;
                    put(e, col / 8 + side, __byte_perm(x[0][0], x[0][1], sel), __byte_perm(x[1][0], x[1][1], sel),
                        __byte_perm(x[2][0], x[2][1], sel), __byte_perm(x[3][0], x[3][1], sel));
                  }
                }
              }
            }
        };
        // tile kt of the item (`left`: and how many after it), its params and first octets asked for before; asks for the
        // next one's, and for the pages of the one after that: nothing of it waits for a round trip to L2. (A loop, not
        // unrolled, here and in the softmax: the warps of an SM run three programs at once, and the whole of it
        // unrolled spent its time waiting for instructions: more than twice as long.)
        Params params, params_next;
        int page = -1, page_next = -1;
        auto begin = [&](int kt, int left) {
          page = octet_page(kt);
          page_next = left > 0 ? octet_page(kt + 1) : -1;
          ask_params(params, kt, page);
          asm volatile("cp.async.wait_all;" ::: "memory");  // (what the last item's end asked for beyond it: zeros)
          for (int i = 0; i < C::AHEAD; ++i) ask(kt, page, i);
        };
        auto two = [&](auto is_v, const Factors& f, uint32_t to, int kt) {
          constexpr int FIRST = decltype(is_v)::value ? 2 : 0;
#pragma unroll 1
          for (int i = FIRST; i < FIRST + 2; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::AHEAD - 1) : "memory");
            write(is_v, f, to, i);
            const bool over = i + C::AHEAD >= 4;
            ask(over ? kt + 1 : kt, over ? page_next : page, (i + C::AHEAD) & 3);
          }
          fence_async_shared();
          __syncwarp();
        };
        // (V: a stage's uses -- key tiles, and per item one epilogue staging -- have positions in
        // order; each of the warps waits for their releases in that order)
        int g = 0;
        uint32_t pos = 0;
        int seen[VST];
        for (int s = 0; s < VST; ++s) seen[s] = 0;
        int prev_stage = -1;
        auto wait_release = [&](uint32_t p) {
          const int s = p % VST, u = p / VST;
          if (seen[s] > u) return true;
          if (!__all_sync(0xffffffffu, wait_free(&bar_vempty[s], u & 1))) return false;
          seen[s] = u + 1;
          return true;
        };
        bool ok = true;
        while (ok && next()) {
          if (seg.n > 0) begin(seg.k0, seg.n - 1);
          for (int t = 0; t < seg.n; ++t, ++g, ++pos) {
            const int kt = seg.k0 + t, left = seg.n - 1 - t, ks = g % KST, vs = pos % VST;
            ask_params(params_next, kt + 1, page_next);
            const int page_after = left > 1 ? octet_page(kt + 2) : -1;
            Exponents exps;
            {
              // (what the stage is not needed for, before it is waited for; all have read tile g - 5's info, the place's last one's long before)
              exps = exponents(params, kt, g);
              const Factors f = factors(std::false_type(), params, exps);
              if (!(ok = __all_sync(0xffffffffu, wait_free(&bar_kempty[ks], ((g / KST) & 1) ^ 1)) != 0)) break;
              if (lane >> 4 == half) {
                // z' 2^8 of key `lane`, high, high and low term of each group (for the high, low and high one of q's sums)
                const uint32_t h = q_half2(f.z[0] / Q_SUM, f.z[1] / Q_SUM);
                const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h));
                const uint32_t l = q_half2(f.z[0] / Q_SUM - hf.x, f.z[1] / Q_SUM - hf.y);
                // h0 h0 | l0 h1 | h1 l1 | 0 0
                st_shared_v4(sKmore(ks) + (quarter * 32 + lane) * 16, __byte_perm(h, h, 0x1010), __byte_perm(l, h, 0x7610),
                             __byte_perm(h, l, 0x7632), 0u);
              }
              two(std::false_type(), f, sK(ks), kt);
            }
            if (lane == 0) mbar_arrive(&bar_kfull[ks]);
            const Factors f = factors(std::true_type(), params, exps);
            if (pos >= (uint32_t)VST && !(ok = wait_release(pos - VST))) break;
            two(std::true_type(), f, sV(vs), kt);
            if (lane == 0) mbar_arrive(&bar_vfull[vs]);
            params = params_next;
            page = page_next;
            page_next = page_after;
          }
          if (!ok) break;
          if (pos >= (uint32_t)VST && !(ok = wait_release(pos - VST))) break;
          if (prev_stage >= 0 && !(ok = wait_release((uint32_t)prev_stage))) break;
          if (lane == 0)
            for (int q = 0; q < NQ; ++q) mbar_arrive(&bar_grant[q]);
          __syncwarp();
          prev_stage = (int)pos;
          ++pos;
        }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp >= C::SOFTMAX_WARPS) {
    regs_decrease<C::REGS_CONTROL>();
    if (BITS && warp == C::KQ_WARP) {
      // ---------------------------------------------------------- Q producer (the codes have their own)
      int j = 0;
      bool ok = true;
      while (ok && next()) {
        if (seg.n == 0) continue;
        for (int q = 0; ok && q < NQ; ++q) {
          if (j > 0 && !(ok = __all_sync(0xffffffffu, wait_free(&bar_qfree[q], (j - 1) & 1)))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar_q[q], (C::NCB * 128u + 16u) * a.RT);
            const int row = seg.s.row0 + a.g.rep.of(seg.x.rho0) + q * a.tpt;
            for (int cb = 0; cb < C::NCB; ++cb) tma_load_4d(sQ(q) + cb * C::CB_BYTES, &tmQ, &bar_q[q], cb * 64, 0, row, seg.head);
            tma_load_4d(sQmore(q), &tmK, &bar_q[q], 0, 0, row, seg.head);
          }
          __syncwarp();
        }
        if (ok) ++j;
      }
      // every issued copy must land before the CTA may exit (those of an item that was given up, for as long as the limit)
      if (j > 0)
        for (int q = 0; q < NQ; ++q) drain(&bar_q[q], (j - 1) & 1);
      if (!ok)
        for (int q = 0; q < NQ; ++q) drain(&bar_q[q], j & 1);
    } else if (!BITS && warp == C::KQ_WARP) {
      // ---------------------------------------------------------- Q / K producer
      int g = 0, j = 0;  // key tiles, items with keys
      int last_k[KST], last_q = -1;
      for (int s = 0; s < KST; ++s) last_k[s] = -1;
      bool ok = true;
      while (ok && next()) {
        if (seg.n == 0) continue;
        int page = page_for(seg.k0);
        for (int t = 0; t < seg.n; ++t, ++g) {
          const int kt = seg.k0 + t, ks = g % KST;
          const int page_next = t + 1 < seg.n ? page_for(kt + 1) : 0;  // (on its way while this tile waits)
          if (!(ok = __all_sync(0xffffffffu, wait_free(&bar_kempty[ks], ((g / KST) & 1) ^ 1)))) break;
          load_tile(sK(ks), &tmK, &bar_kfull[ks], kt, page);
          last_k[ks] = g / KST;
          page = page_next;
          if (t == 0) {
            for (int q = 0; ok && q < NQ; ++q) {
              if (j > 0 && !(ok = __all_sync(0xffffffffu, wait_free(&bar_qfree[q], (j - 1) & 1)))) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(&bar_q[q], C::NCB * 128u * a.RT);
                for (int cb = 0; cb < C::NCB; ++cb)
                  tma_load_4d(sQ(q) + cb * C::CB_BYTES, &tmQ, &bar_q[q], cb * 64, 0,
                              seg.s.row0 + a.g.rep.of(seg.x.rho0) + q * a.tpt, seg.head);
              }
              __syncwarp();
            }
            if (!ok) break;
            last_q = j;
          }
        }
        ++j;
      }
      // every issued copy must land before the CTA may exit
      for (int s = 0; s < KST; ++s)
        if (last_k[s] >= 0) drain(&bar_kfull[s], last_k[s] & 1);
      if (last_q >= 0)
        for (int q = 0; q < NQ; ++q) drain(&bar_q[q], last_q & 1);
    } else if (!BITS && warp == C::V_WARP) {
      // ---------------------------------------------------------- V producer
      // (a stage's uses -- key tiles, and per item one epilogue staging -- have positions in
      // order, and this warp alone waits for their releases, in that order)
      uint32_t pos = 0;
      int seen[VST], loads[VST];
      for (int s = 0; s < VST; ++s) { seen[s] = 0; loads[s] = 0; }
      int prev_stage = -1;
      bool ok = true;
      auto wait_release = [&](uint32_t p) {
        const int s = p % VST, u = p / VST;
        if (seen[s] > u) return true;
        if (!__all_sync(0xffffffffu, wait_free(&bar_vempty[s], u & 1))) return false;
        seen[s] = u + 1;
        return true;
      };
      while (ok && next()) {
        int page = seg.n > 0 ? page_for(seg.k0) : 0;
        for (int t = 0; t < seg.n; ++t, ++pos) {
          const int kt = seg.k0 + t;
          const int page_next = t + 1 < seg.n ? page_for(kt + 1) : 0;
          if (pos >= (uint32_t)VST && !(ok = wait_release(pos - VST))) break;
          load_tile(sV(pos % VST), &tmV, &bar_vfull[pos % VST], kt, page);
          ++loads[pos % VST];
          page = page_next;
        }
        if (!ok) break;
        if (pos >= (uint32_t)VST && !(ok = wait_release(pos - VST))) break;
        if (prev_stage >= 0 && !(ok = wait_release((uint32_t)prev_stage))) break;
        if (lane == 0)
          for (int q = 0; q < NQ; ++q) mbar_arrive(&bar_grant[q]);
        __syncwarp();
        prev_stage = (int)pos;
        ++pos;
      }
      for (int s = 0; s < VST; ++s)
        if (loads[s] > 0) drain(&bar_vfull[s], (loads[s] - 1) & 1);
    } else if (warp == C::MMA_WARP) {
      // ---------------------------------------------------------- MMA issuer
      int g = 0, j = 0;
      uint32_t pos = 0;
      while (next()) {
        const int n = seg.n;
        if (n == 0) { pos += 1; continue; }
        const int k0 = g % KST;
        for (int q = 0; q < NQ; ++q) {
          named_bar_sync(C::RELAY_BAR, 64);
          tc_fence_after();
          if (elect_one()) {
            issue_qk<C>(tmem + C::s_col(q), sQ(q), sK(k0), sQmore(q), sKmore(k0), sbase + C::ZERO_OFF);
            tc_commit(&bar_s[q]);
            if (n == 1) tc_commit(&bar_qfree[q]);
          }
          __syncwarp();
        }
        if (elect_one()) tc_commit(&bar_kempty[k0]);
        __syncwarp();
        for (int t = 0; t < n; ++t, ++g, ++pos) {
          const int vs = pos % VST, ks = (g + 1) % KST;
          const bool more = t + 1 < n;
          named_bar_sync(C::RELAY_BAR, 64);  // V_g (and K_{g+1}) are in shared memory
          for (int q = 0; q < NQ; ++q) {
            named_bar_sync(1 + q, 128 + 32);  // P_q(g) is in TMEM
            tc_fence_after();
            if (elect_one()) {
              issue_pv<C, TERMS>(tmem + C::o_col(q), tmem + C::s_col(q), sV(vs), t > 0);
              if (more) {
                issue_qk<C>(tmem + C::s_col(q), sQ(q), sK(ks), sQmore(q), sKmore(ks), sbase + C::ZERO_OFF);
                tc_commit(&bar_s[q]);
                if (t + 2 == n) tc_commit(&bar_qfree[q]);
              } else {
                tc_commit(&bar_o[q]);
              }
            }
            __syncwarp();
          }
          if (elect_one()) {
            tc_commit(&bar_vempty[vs]);
            if (more) tc_commit(&bar_kempty[ks]);
          }
          __syncwarp();
        }
        pos += 1;
        ++j;
      }
      if (j > 0 && elect_one()) {
        tc_commit(&bar_drain);  // no MMA may still be running when TMEM is released
        drain(&bar_drain, 0);
      }
      __syncwarp();
    } else if (warp == C::RELAY_WARP) {
      // ---------------------------------------------------------- load relay
      bool ok = true;
      int g = 0, j = 0;
      uint32_t pos = 0;
      int vc[VST];
      for (int s = 0; s < VST; ++s) vc[s] = 0;
      while (next()) {
        const int n = seg.n;
        if (n == 0) { pos += 1; continue; }
        for (int q = 0; q < NQ; ++q) {
          if (ok)
            ok = __all_sync(0xffffffffu,
                            wait(&bar_q[q], j & 1) && (q > 0 || wait(&bar_kfull[g % KST], (g / KST) & 1)));
          named_bar_sync(C::RELAY_BAR, 64);
        }
        for (int t = 0; t < n; ++t, ++g, ++pos) {
          const bool more = t + 1 < n;
          const int vs = pos % VST;
          if (ok)
            ok = __all_sync(0xffffffffu, wait(&bar_vfull[vs], vc[vs] & 1) &&
                                             (!more || wait(&bar_kfull[(g + 1) % KST], ((g + 1) / KST) & 1)));
          ++vc[vs];
          const int end = seg.s.len - (seg.k0 + t) * BLOCK_N;  // tokens from here on are past the sequence
          if (!BITS && ok && end < BLOCK_N) {
            for (int i = end * 8 + lane; i < BLOCK_N * 8; i += 32)
              for (int cb = 0; cb < C::NCB; ++cb) st_shared_v4(sV(vs) + cb * C::CB_BYTES + i * 16, 0, 0, 0, 0);
            fence_async_shared();
            __syncwarp();
          }
          named_bar_sync(C::RELAY_BAR, 64);
        }
        pos += 1;
        ++j;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    regs_increase<C::REGS_SOFTMAX>();
    const int q = warp / 4, wq = warp % 4;
    const int r_in = wq * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t s_addr = lane_addr + C::s_col(q);
    const uint32_t o_addr = lane_addr + C::o_col(q);
    const float sl2 = a.sl2;
    bool ok = true, live = true;  // epilogues are granted; the issuer goes on
    int g = 0, j = 0, k = 0;
    uint32_t pos = 0;
    // One warp gives the epilogue's stage back, once all have read their parts of it: after its
    // next hand-off, so that the next P does not wait for it.
    bool pending = false;
    int pend_slot = 0, pend_item = 0;
    auto release = [&]() {
      if (ok) ok = __all_sync(0xffffffffu, wait(&bar_join, pend_item & 1));
      if (ok && lane == 0) mbar_arrive(&bar_vempty[pend_slot]);
      __syncwarp();
      pending = false;
    };
    for (; next(); ++k) {
      const int n = seg.n;
      // this tile's rows: rho0 + r, r < rows; row r is token r / rep of the tile
      const int rho0 = seg.x.rho0 + q * a.RT;
      const int rows = max(0, min(a.RT, seg.x.rows - q * a.RT));
      const int p0 = seg.s.len - seg.s.n + a.g.rep.of(rho0);  // position of its first token
      const int p1 = p0 + a.g.rep.of(max(0, rows - 1));
      const int p = p0 + a.g.rep.of(r_in);
      const int last = seg.s.len - 1;
      const int hi_i = a.g.causal ? min(p, last) : last;
      const int lo_i = a.g.window > 0 ? p - a.g.window + 1 : 0;
      const int in_hi = a.g.causal ? min(p0, last) : last;  // keys that every row sees
      const int in_lo = a.g.window > 0 ? p1 - a.g.window + 1 : 0;
      float m = BITS && r_in >= rows ? 0.f : -FLT_MAX, l = 0.f;
      // codes: the row's factor, and the exponent that the probabilities are taken against (O is O * 2^v_ref)
      float qf = 0.f, v_ref = 0.f;
      if (BITS && r_in < rows) {
        const int token = a.g.rep.of(rho0 + r_in);
        qf = a.qf[(size_t)(seg.s.row0 + token) * a.H + seg.head * a.g.rep.d + rho0 + r_in - token * a.g.rep.d];
      }
      for (int t = 0; t < n; ++t, ++g) {
        if (live) live = __all_sync(0xffffffffu, wait_issuer(&bar_s[q], g & 1));
        if (!live) {
          named_bar_sync(1 + q, 128 + 32);  // every round is joined, whatever happens
          if (pending) release();
          continue;
        }
        tc_fence_after();
        if constexpr (BITS != 0) {
          const float2* const info = info_sh[g % TILE_INFO];
          const int c0 = (seg.k0 + t) * BLOCK_N;
          const bool edge = c0 < in_lo || c0 + BLOCK_N - 1 > in_hi;
          const float v_top = fmaxf(fmaxf(info[0].y, info[1].y), fmaxf(info[2].y, info[3].y));
          auto rescale = [&](float by) {  // of O's row
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(o_addr + c * 32, r);
#pragma unroll
              for (int kk = 0; kk < 32; ++kk) r[kk] = __float_as_uint(__uint_as_float(r[kk]) * by);
              tmem_st32(o_addr + c * 32, r);
            }
            tmem_st_wait();  // (a tile may do it three times: a load is not ordered behind a store by itself)
          };
          // (2^8 of a probability and 2^6 of V's exponent beyond v_ref: P is 2^14 at most. v_ref is the row's, and goes by
          // the keys that it sees: of 32 that share an exponent those of which it sees one)
          if (__any_sync(0xffffffffu, t == 0 || v_top > v_ref + 6.f)) {
            float v_row = -106.f;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              const float y = info[b].y;
              if (y < OWN / 2) {
                if (c0 + 32 * b <= hi_i && c0 + 32 * b + 31 >= lo_i) v_row = fmaxf(v_row, y);
              } else {
                const uint32_t* const keys = &keys_sh[g % TILE_INFO][32 * b];
#pragma unroll 1
                for (int kk = max(0, lo_i - c0 - 32 * b); kk <= min(31, hi_i - c0 - 32 * b); ++kk)
                  v_row = fmaxf(v_row, (float)q_exponent(q_scale(keys[kk])));
                __syncwarp();  // (rows see different keys: together again for tensor memory)
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                  uint32_t r[16];
                  tmem_ld16(s_addr + 32 * b + c, r);
#pragma unroll
                  for (int kk = 0; kk < 16; ++kk) r[kk] = __float_as_uint(__uint_as_float(r[kk]) * q_offset(keys[c + kk]));
                  tmem_st16(s_addr + 32 * b + c, r);
                }
                tmem_st_wait();
              }
            }
            v_row -= 5.f;  // (room for one more: what is under 2^-30 of the largest V is lost in P, not 2^-25)
            const bool more = t == 0 || v_row > v_ref + 1.f;
            if (t > 0 && __any_sync(0xffffffffu, more)) rescale(more ? ex2(v_ref - v_row) : 1.f);
            if (more) v_ref = v_row;
          }
          // 64 keys at a time, in a loop (see the code warps), P in the place of scores that are read. m moves by whole
          // powers of two: where it does, O, l and what is written of P follow exactly.
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const float2 i0 = info[2 * h], i1 = info[2 * h + 1];
            float s[64];
            {
              uint32_t v[32], u[32];
              tmem_ld32x2(s_addr + h * 64, s_addr + h * 64 + 32, v, u);
#pragma unroll
              for (int kk = 0; kk < 32; ++kk) {
                s[kk] = __uint_as_float(v[kk]);
                s[32 + kk] = __uint_as_float(u[kk]);
              }
            }
            if (edge) mask_outside<64>(s, lo_i - c0 - 64 * h, hi_i - c0 - 64 * h);
            // (positive whatever the row: a masked score is -infinity times it)
            float kc[2] = {fmaxf(qf * i0.x, FLT_MIN), fmaxf(qf * i1.x, FLT_MIN)};
            // (far below that, P is 0 in fp16; above it no key that the row sees)
            const float up[2] = {fminf(fmaxf(i0.y - v_ref, -60.f), 6.f), fminf(fmaxf(i1.y - v_ref, -60.f), 6.f)};
            float mt = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float mx[4];
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mx[kk] = max3(s[32 * b + kk], s[32 * b + 4 + kk], s[32 * b + 8 + kk]);
#pragma unroll
              for (int k = 12; k < 28; k += 8)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mx[kk] = max3(mx[kk], s[32 * b + k + kk], s[32 * b + k + 4 + kk]);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mx[kk] = fmaxf(mx[kk], s[32 * b + 28 + kk]);
              mt = fmaxf(mt, fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * kc[b]);
            }
            // (each row for itself: no row's bits depend on another's)
            const bool grow = r_in < rows && mt > m + RESCALE_THRESHOLD;
            float less = m;  // (what is to be taken off in one operation with the product)
            if (__any_sync(0xffffffffu, grow || fabsf(m) > Q_LARGE)) {
              const float m_new = grow ? ceilf(mt) : m, corr = ex2(m - m_new);
              l *= corr;
              if (t > 0) rescale(corr);
              if (h > 0) {
                // (P is up to 2^14, so corr is not to be lost before it: 2^-14 of it, and the rest)
                const float most = fmaxf(corr, 0x1p-14f), rest = corr * (1.f / most);
                const uint32_t by = pack_half2(most, most), by2 = pack_half2(rest, rest);
                tmem_st_wait();
                uint32_t r[32];
                tmem_ld32(s_addr, r);
#pragma unroll
                for (int kk = 0; kk < 32; ++kk) r[kk] = q_mul2(q_mul2(r[kk], by), by2);
                tmem_st32(s_addr, r);
              }
              less = m = m_new;
              if (fabsf(m) > Q_LARGE) {
#pragma unroll
                for (int kk = 0; kk < 64; ++kk) s[kk] = __fsub_rn(__fmul_rn(s[kk], kc[kk / 32]), m);
                kc[0] = kc[1] = 1.f;
                less = 0.f;
              }
              __syncwarp();
            }
            uint32_t pk[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float2 by = make_float2(kc[b], kc[b]), off = make_float2(up[b] - less, up[b] - less);
              float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int kk = 0; kk < 16; ++kk) {
                const float2 x = fma2(make_float2(s[32 * b + 2 * kk], s[32 * b + 2 * kk + 1]), by, off);
                const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                ls[kk & 1] = add2(ls[kk & 1], pp);
                pk[16 * b + kk] = pack_half2(pp.x, pp.y);
              }
              l = fmaf((ls[0].x + ls[1].x) + (ls[0].y + ls[1].y), ex2(-up[b]), l);
            }
            tmem_st32(s_addr + h * 32, pk);
          }
          // P of keys that have exponents of their own, which were taken to be 6 beyond v_ref
          if (__any_sync(0xffffffffu, v_top > OWN / 2)) {
            tmem_st_wait();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              if (info[b].y < OWN / 2) continue;
              const uint32_t* const keys = &keys_sh[g % TILE_INFO][32 * b];
              uint32_t r[16];
              tmem_ld16(s_addr + 16 * b, r);
#pragma unroll
              for (int kk = 0; kk < 16; ++kk) {
                auto by = [&](int k) { return ex2(fminf((float)q_exponent(q_scale(keys[k])) - 6.f - v_ref, 0.f)); };
                r[kk] = q_mul2(r[kk], q_half2(by(2 * kk), by(2 * kk + 1)));
              }
              tmem_st16(s_addr + 16 * b, r);
            }
          }
        } else {
        float s[128];
        {
          uint32_t v0[32], v1[32], v2[32], v3[32];
          tmem_ld32x4(s_addr, s_addr + 32, s_addr + 64, s_addr + 96, v0, v1, v2, v3);
#pragma unroll
          for (int kk = 0; kk < 32; ++kk) {
            s[kk] = __uint_as_float(v0[kk]);
            s[32 + kk] = __uint_as_float(v1[kk]);
            s[64 + kk] = __uint_as_float(v2[kk]);
            s[96 + kk] = __uint_as_float(v3[kk]);
          }
        }
        const int c0 = (seg.k0 + t) * BLOCK_N;
        if (c0 < in_lo || c0 + BLOCK_N - 1 > in_hi) mask_outside<128>(s, lo_i - c0, hi_i - c0);
        float mx[8];
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mx[kk] = max3(s[kk], s[8 + kk], s[16 + kk]);
#pragma unroll
        for (int c = 24; c < 120; c += 16)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mx[kk] = max3(mx[kk], s[c + kk], s[c + 8 + kk]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mx[kk] = fmaxf(mx[kk], s[120 + kk]);
        const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sl2;
        // (rows past the item's have no say: they are another sequence's, or whatever lay in the stage, and a
        // maximum that moved earlier would round the others' probabilities differently)
        if (__any_sync(0xffffffffu, r_in < rows && mt > m + RESCALE_THRESHOLD)) {
          const float m_new = fmaxf(m, mt);
          const float corr = ex2(m - m_new);
          l *= corr;
          if (t > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(o_addr + c * 32, r);
#pragma unroll
              for (int kk = 0; kk < 32; ++kk) r[kk] = __float_as_uint(__uint_as_float(r[kk]) * corr);
              tmem_st32(o_addr + c * 32, r);
            }
          }
          m = m_new;
        }
        const float2 sl2x2 = make_float2(sl2, sl2), nmx2 = make_float2(-m, -m);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
          uint32_t lo[TERMS > 1 ? 32 : 1];
#pragma unroll
          for (int kk = 0; kk < 32; ++kk) {
            const float2 x = fma2(make_float2(s[c * 64 + 2 * kk], s[c * 64 + 2 * kk + 1]), sl2x2, nmx2);
            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
            ls[kk & 1] = add2(ls[kk & 1], pp);
            pk[kk] = pack_bf2(pp.x, pp.y);
            if constexpr (TERMS > 1)
              lo[kk] = pack_bf2(pp.x - __uint_as_float(pk[kk] << 16), pp.y - __uint_as_float(pk[kk] & 0xffff0000u));
          }
          tmem_st32(s_addr + c * 32, pk);
          if constexpr (TERMS > 1) tmem_st32(s_addr + 64 + c * 32, lo);
        }
        l += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
        }
        tmem_st_wait();
        tc_fence_before();
        named_bar_arrive(1 + q, 128 + 32);
        if (pending) release();
      }
      pos += n;
      if (n > 0) {
        if (live) live = __all_sync(0xffffffffu, wait_issuer(&bar_o[q], j & 1));
        tc_fence_after();
        ++j;
      }
      if (pending) release();
      ok = ok && live;
      // ---- epilogue, staged in this tile's half of the item's V ring stage
      const int slot = pos % VST;
      if (ok) ok = __all_sync(0xffffffffu, wait(&bar_grant[q], k & 1));
      const uint32_t stage = sV(slot) + (uint32_t)warp * C::EPI_BOX;
      const bool whole = seg.starts && seg.ends;
      if (ok) {
        const int warp_rows = rows - wq * 32;  // rows of this warp's 32 that exist
        // rows go to O, or, of a part, to its slot: `at(r)` is row r's place in either
        const size_t slot_row = (size_t)(2 * blockIdx.x + seg.slot) * a.g.R + q * a.RT;
        auto at = [&](int r) {
          if (!whole) return slot_row + r;
          const int token = a.g.rep.of(rho0 + r);
          return (size_t)(seg.s.row0 + token) * a.H + seg.head * a.g.rep.d + rho0 + r - token * a.g.rep.d;
        };
        char* const to = whole ? static_cast<char*>(a.O) : reinterpret_cast<char*>(a.part.O);
        const bool bf = whole && a.out_bf16;
        const int cols = whole ? a.c.D : D;
        const size_t row_bytes = (size_t)cols * (bf ? 2 : 4);
        auto ptr = [&](int r) -> char* { return r < warp_rows ? to + at(wq * 32 + r) * row_bytes : nullptr; };
        const float inv = (!whole ? 1.f : l == 0.f ? 0.f : __fdividef(1.f, l)) * (BITS ? ex2(v_ref) : 1.f);  // (NaN stays)
        if (r_in < rows) {
          if (whole) a.LSE[at(r_in)] = l == 0.f ? -INFINITY : (m + __log2f(l)) * LN2;
          else a.part.ml[at(r_in)] = make_float2(m, l);
        }
        if (bf) store_rows<D, true>(o_addr, n > 0, inv, stage, cols, ptr);
        else store_rows<D, false>(o_addr, n > 0, inv, stage, cols, ptr);
        if (!whole && threadIdx.x == 0)
          a.part.left[2 * blockIdx.x + seg.slot] = {
              (seg.starts ? PART_STARTS : 0) | (seg.ends ? PART_ENDS : 0), seg.s.row0, seg.x.rho0,
              seg.x.rows, seg.head, walk.p.ender, {0, 0}};
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bar_join);  // this warp has read its part of the stage
      if (q == NQ - 1 && wq == 0) {
        pending = true;
        pend_slot = slot;
        pend_item = k;
      }
      pos += 1;
    }
    if (pending) release();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, int TERMS, int BITS>
fa_status run(TilesArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  using C = TilesCfg<D, BITS>;
  auto* kernel = attend_tiles_kernel<D, TERMS, BITS>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return failed();
  const int ctas = host::sm_count();
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas, a.g.R, D), s) != cudaSuccess) return failed();
  a.part = partials_at(w, ctas, a.g.R, D);
  fa_status st;
  {
    host::KernelTimer t(BITS ? "qattend_tiles" : "attend_tiles", s);
    if (BITS) st = launch_programmatic_smem(kernel, ctas, C::THREADS, C::SMEM, s, q, k, v, a) == cudaSuccess ? FA_OK : failed();
    else st = launch(kernel, ctas, C::THREADS, C::SMEM, s, q, k, v, a);
  }
  if (st == FA_OK) {
    const JoinArgs j = {a.part, a.O, a.LSE, ctas, 1, a.g.R, D, a.H, a.c.D, a.out_bf16, a.g.rep};
    st = launch_join_tall(j, s);
  }
  if (host::scratch_free(w, s) != cudaSuccess) st = failed();
  return st;
}

// q as [HKV][T][rep][D] (`columns` D; or 8 more, of 16 bytes to a row and without a swizzle)
bool map_q(CUtensorMap* m, const TilesArgs& a, const void* q, long long token, long long head, int columns) {
  const int rep = a.g.rep.d;
  const uint64_t qd[4] = {(uint64_t)columns, (uint64_t)rep, (uint64_t)a.T, (uint64_t)a.c.HKV};
  const uint64_t qs[3] = {(uint64_t)head * 2, (uint64_t)token * 2, (uint64_t)head * rep * 2};
  const uint32_t qb[4] = {columns == 8 ? 8u : 64u, (uint32_t)rep, (uint32_t)a.tpt, 1};
  return host::encode_tiled_4d(m, q, qd, qs, qb, columns != 8);
}

TilesArgs args_of(void* O, float* LSE, const int* cu, const int* slots, const fakv_cache& c, const fakv_tokens& p) {
  TilesArgs a = {};
  const int rep = p.H / c.HKV;
  a.c = c;
  a.O = O;
  a.LSE = LSE;
  a.cu = cu;
  a.slots = slots;
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.shift = log2_of(c.page_size);
  a.tpt = 128 / rep;
  a.RT = a.tpt * rep;
  a.box = std::min(c.page_size, BLOCK_N);
  a.boxes = BLOCK_N / a.box;
  a.g = {div_by(rep), 2 * a.RT, log2_of(BLOCK_N), 3, 2, p.causal, p.window};  // (an item's beginning and end take three units' time)
  a.sl2 = p.scale * LOG2E;
  a.out_bf16 = p.out_dtype == FA_BF16;
  a.limit_ns = WAIT_LIMIT_NS;
  return a;
}

}  // namespace

fa_status launch_attend_tiles(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                              const fakv_cache& c, const fakv_tokens& p, cudaStream_t s) {
  if (host::sm_count() > TALL_CTAS) return FA_ERR_UNSUPPORTED;
  TilesArgs a = args_of(O, LSE, cu, slots, c, p);
  const uint64_t d = c.D, b2 = 2;
  CUtensorMap mq, mk, mv;
  // the pages as [page][head][token][D]
  const uint64_t kd[4] = {d, (uint64_t)c.page_size, (uint64_t)c.HKV, (uint64_t)c.num_pages};
  const uint64_t ks[3] = {(uint64_t)c.token_stride * b2, (uint64_t)c.head_stride * b2, (uint64_t)c.page_stride * b2};
  const uint32_t kb[4] = {64, (uint32_t)a.box, 1, 1};
  const long long plane = p.plane * c.plane_stride * 2;
  if (!map_q(&mq, a, q, p.q_token, p.q_head, c.D) || !host::encode_tiled_4d(&mk, static_cast<const char*>(c.K) + plane, kd, ks, kb) ||
      !host::encode_tiled_4d(&mv, static_cast<const char*>(c.V) + plane, kd, ks, kb))
    return FA_ERR_UNSUPPORTED;
  if (a.out_bf16) return c.D <= 64 ? run<64, 1, 0>(a, mq, mk, mv, s) : run<128, 1, 0>(a, mq, mk, mv, s);
  return c.D <= 64 ? run<64, 2, 0>(a, mq, mk, mv, s) : run<128, 2, 0>(a, mq, mk, mv, s);
}

fa_status launch_qattend_tiles(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                               const QCache& qc, const fakv_tokens& p, cudaStream_t s) {
  if (host::sm_count() > TALL_CTAS) return FA_ERR_UNSUPPORTED;
  TilesArgs a = args_of(O, LSE, cu, slots, qc.c, p);
  a.qc = qc;
  a.raised = Q_RAISED;
  const int D = qc.c.D, rows = p.T * p.H;
  const size_t row_bytes = ((size_t)rows * D * 2 + 255) & ~(size_t)255, more_bytes = ((size_t)rows * 16 + 255) & ~(size_t)255;
  void* w = nullptr;
  if (host::scratch_alloc(&w, row_bytes + more_bytes + (size_t)rows * 4, s) != cudaSuccess) return failed();
  char* const more = static_cast<char*>(w) + row_bytes;
  float* const qf = reinterpret_cast<float*>(more + more_bytes);
  a.qf = qf;
  CUtensorMap mq, mm;
  fa_status st = map_q(&mq, a, w, (long long)p.H * D, D, D) && map_q(&mm, a, more, (long long)p.H * 8, 8, 8) ? FA_OK : FA_ERR_UNSUPPORTED;
  if (st == FA_OK) {
    host::KernelTimer t("qattend_q", s);
    st = launch(qattend_q_kernel, (rows + QROWS_THREADS / 16 - 1) / (QROWS_THREADS / 16), QROWS_THREADS, 0, s,
                static_cast<const __nv_bfloat16*>(q), p.q_token, p.q_head, rows, div_by(p.H), D, qc.groups, a.sl2, qc.bits == 4,
                static_cast<uint16_t*>(w), reinterpret_cast<uint4*>(more), qf);
  }
  if (st == FA_OK && qc.bits == 4) st = D <= 64 ? run<64, 1, 4>(a, mq, mm, mm, s) : run<128, 1, 4>(a, mq, mm, mm, s);
  else if (st == FA_OK) st = D <= 64 ? run<64, 1, 8>(a, mq, mm, mm, s) : run<128, 1, 8>(a, mq, mm, mm, s);
  if (host::scratch_free(w, s) != cudaSuccess) st = failed();
  return st;
}

unsigned int read_and_clear_kv_status(cudaError_t* err) {
  unsigned int v = 0, zero = 0;
  *err = cudaMemcpyFromSymbol(&v, g_kv_status, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(zero));
  return v;
}

}  // namespace kv
}  // namespace fa
