// kv_qrows.cu -- attention over the cache in 4 or 8 bits for few rows per sequence (decoding), and for
// fp32 queries: codes streamed once, made fp16 in registers, mma.sync.
//
// Workers, parts and joins are those of kv_rows.cu. A page of a head is one block of memory, its codes one
// after another: the copy engine brings a step's 64 or 32 keys in a few copies (two a page), which the lanes issue
// whose pages they are, and every wait for one has a limit. With s, z of a key's group g and codes
// c = centre + x (centre 8 or 128), its K and V are s x + z', z' = z + centre s, so that
//
//   scores  S = sum_g s_g (sum_{d in g} q_d c_d) + z_g (sum_{d in g} q_d): codes are exact fp16
//           operands, 2^-24 c, the numbers that fp16 has below its normal ones: an and of the word makes two, and
//           there is no constant to take off, which for 1024 + c left LSEs up to 2.8e-6 of themselves off and took 144 us where
//           this took 135; a key's scales come after the products, in fp32. (O in fp32: x, which costs an addition
//           a pair.) q times a power of two per row that brings its largest value to 2^14 is fp16 too, exactly but for
//           what is 2^-28 of that
//   O^T     O_d = sum_k (p_k s_k) x_kd + sum_k p_k z'_k: the scales enter the probabilities, times a power
//           of two that keeps the largest scale that the row has seen at most 2^6; the offsets are one more sum
//           per row and group. p s is one fp16 term where O is bf16 (2^-11 of itself, an eighth of O's
//           own rounding), two (2^-22) where O is fp32; what is below 2^-30 of the largest p s rounds to
//           2^-40 of it. (A power of two to a row: with one for an item, a key that a row does not see and whose V is
//           2^31 times as large took from it all that codes stand for)
//
// so nothing of the cache is rounded again. A code costs about an instruction (kv_quant.cuh):
//   K  columns are what is summed over, in any order: a thread takes the 8 (4) columns of one
//      32-bit word of its key, and q's fragments are laid out to match
//   V  keys are summed over, two of each register: the cache holds the codes of two tokens side by side,
//      so that every pair is one column of two keys
//
// Measured (device, data in L2 where they fit; floor: bytes at the measured copy rate): 64 sequences of up to 16384 tokens in
// 4 bits, D 128, 130 us (floor 89); 32 of up to 8192 in 8 bits 60 (42; 70 cold); one of 1021 12; 16 of up to 8192
// with 4 drafted tokens each 41 (12; two warps to a scheduler, 37 % of issue). Not HBM but the instructions that make numbers of codes bound it: 304 to 16 keys of
// a head (a half of them on the ALU), 56 % of what the warps' schedulers can issue, with three warps to each: more do not fit
// (128 registers for 16 warps an SM spilled: 153 us). Sixteen rows take those instructions once for two rows' tiles;
// with more rows they are taken again for every sixteen, and kv_tiles.cu takes over where that costs more. 64 keys to a step
// where there is room: 153 -> 140 us when that was done. V's codes are x and not c: their sums over thousands of keys
// would lose to c's mean what the tensor cores cut off at each product (c, and the mean taken off by a second product: 137).
#include <algorithm>
#include "kv_quant.cuh"
#include "kv_rows.cuh"

namespace fa {
namespace kv {

static __device__ unsigned int g_kvq_status = 0;

namespace {

struct QRowsArgs {
  fakv_cache c;
  QCache qc;
  const void* q;
  void* O;
  float* LSE;
  const int* cu;
  const int* slots;
  int B, T, H, shift;
  long long q_token, q_head;
  Geo g;
  float sl2;  // scale * log2(e)
  uint32_t raised;  // Q_RAISED
  int out_bf16;
  int run_shift;  // log2 of the keys of a run: of a step, in one page, one after another in memory
  Partials part;
};

template <typename E, bool OUT_BF, int BITS, int D, int NG_, int NTR>
struct QRowsCfg {
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int TERMS = F32 ? 2 : 1;       // fp16 terms of q
  static constexpr int PT = OUT_BF ? 1 : 2;       // and of P times a key's scale
  static constexpr int R = 8 * NTR;               // rows of an item
  static constexpr int CH = D * BITS / 128;       // 16-byte chunks of a key's codes
  static constexpr int NG = NG_;                  // groups of a key
  static constexpr int KS = D / 16;               // k16 steps of q
  static constexpr int GROUP = NTR == 1 && OUT_BF && D * BITS <= 512 ? 64 : 32;  // keys of a step
  static constexpr int GROUP_SHIFT = GROUP == 64 ? 6 : 5;
  static constexpr int KT = GROUP / 16;
  static constexpr int CODES = GROUP * CH * 16;
  static constexpr int SLOT = CODES + GROUP * NG * 4;  // K (or V) of a step
  static constexpr bool Q_REGS = NTR == 1 && !F32;     // q's fragments stay in registers
  static constexpr int Q_BYTES = Q_REGS ? 0 : NTR * TERMS * (KS / 2) * 512;
  static constexpr int OS = D + 4;                // floats of a row of O in shared memory (bank spread)
  static constexpr int CTAS_PER_SM = Q_REGS ? 3 : 2;
  static constexpr int ROOM = CTAS_PER_SM == 3 ? 18432 : 28160;
  static constexpr int NP = std::min(6, (ROOM - Q_BYTES) / (2 * SLOT));  // steps of the ring
  static constexpr int WARP_BYTES = std::max({NP * 2 * SLOT + Q_BYTES, R * OS * 4, 16512});
  static constexpr int SMEM = WARPS * WARP_BYTES;
  static_assert(NP >= 2 && WARP_BYTES % 128 == 0 && SLOT % 128 == 0 && Q_BYTES % 128 == 0, "the ring");
  static_assert(SMEM >= 4 * 16385, "the plan's scratch");
  static constexpr int STATIC = (int)sizeof(PlanShared<NTHREADS, WARPS>) + WARPS * (R * 8 + 20 + NP * 8) + 8;
  static_assert(CTAS_PER_SM * (SMEM + (STATIC + 1023) / 1024 * 1024 + 1024) <= 228 * 1024, "shared memory of the CTAs of an SM");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// a and b as fp16 (low, high); rest: what is left of them
__device__ __forceinline__ uint32_t half2_of(float a, float b, float2* rest = nullptr) {
  const __half2 h = __floats2half2_rn(a, b);
  if (rest) {
    const float2 f = __half22float2(h);
    *rest = make_float2(a - f.x, b - f.y);
  }
  return *reinterpret_cast<const uint32_t*>(&h);
}
// bytes (a multiple of 16, all of it aligned to 16) into shared memory, counted by `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar)) : "memory");
}
template <typename E, bool OUT_BF, int BITS, int D, int NG_, int NTR>
__global__ void __launch_bounds__(NTHREADS, QRowsCfg<E, OUT_BF, BITS, D, NG_, NTR>::CTAS_PER_SM)
    qattend_rows_kernel(const __grid_constant__ QRowsArgs a) {
  using C = QRowsCfg<E, OUT_BF, BITS, D, NG_, NTR>;
  constexpr int CH = C::CH, R = C::R, NP = C::NP, GROUP = C::GROUP, KT = C::KT, NG = C::NG, KS = C::KS;
  constexpr int TERMS = C::TERMS, PT = C::PT;
  // K's codes: 2^-24 times the code (q_small), or, where O is fp32, centred: an instruction more, and sums of an eighth
  constexpr bool CENTRED = !OUT_BF;
  constexpr float CENTRE = BITS == 4 ? 8.f : 128.f;
  constexpr float NO_LIFT = 0x1p126f;
  constexpr int VT = BITS == 4 ? 2 : 1;  // output tiles of a chunk: code pairs 2 t and 2 t + 1 of a word of V
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ PlanShared<NTHREADS, WARPS> plan;
  __shared__ Ends<R> ends_sh;
  __shared__ __align__(8) uint64_t bars[WARPS][NP];  // of a step's K and V
  __shared__ int abort_sh;
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, oct = lane >> 2;  // mma fragments: columns 2 quad, 2 quad + 1; row oct
  const fakv_cache& c = a.c;
  const Geo& g = a.g;
  const int chunks = a.qc.chunks;
  const int runs_shift = C::GROUP_SHIFT - a.run_shift;  // log2 of the runs of a step
  const uint32_t run_codes = chunks * 16 << a.run_shift, run_params = NG * 4 << a.run_shift;  // bytes
  if (lane < NP) ptx::mbar_init(&bars[warp][lane], 1 << runs_shift);
  if (tid == 0) abort_sh = 0;
  ptx::fence_mbar_init();
  __syncthreads();
  Seq seq;
  const Part part = find_part<NTHREADS, WARPS>(g, c, a.cu, a.slots, a.B, a.T, reinterpret_cast<int*>(smem), plan, seq);
  Walk walk(part, seq);
  const int worker = blockIdx.x * WARPS + warp;
  if (lane < 2) a.part.left[2 * worker + lane].flags = 0;
  if (lane == 0) ends_sh.item[warp] = make_int4(walk.p.b, walk.p.tile, walk.p.head, 2);
  uint8_t* const mine = smem + warp * C::WARP_BYTES;
  const uint32_t sq = ptx::smem_u32(mine);
  // params of key 16 kt + 8 e + oct
  auto params = [&](const uint8_t* slot, int kt, int e, uint32_t (&p)[NG]) {
    const uint8_t* const at = slot + C::CODES + (kt * 16 + e * 8 + oct) * NG * 4;
    if constexpr (NG == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      p[0] = v.x;
      p[1] = v.y;
    } else {
      p[0] = *reinterpret_cast<const uint32_t*>(at);
    }
  };
  const long long v_minus_k = a.qc.V - a.qc.K;
  int ring = 0, parity = 0;  // the next step's place, and how often (mod 2) it was filled before
  auto wait = [&](uint64_t* bar) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, &abort_sh, &g_kvq_status, DEV_TIMEOUT, WAIT_LIMIT_NS)) != 0;
  };
  bool ok = true;
  Seg seg = {};
  Finish fin;
  bool held = false;  // the worker's only item, not done whole: its result waits for the others'

  while (walk.next(g, c, a.cu, a.slots, a.T, seg)) {
    const Seq& s = seg.s;
    const Tile& x = seg.x;

    // ---- where the next 32 runs of keys lie (a run: keys of a step that lie in one page, one after
    // another), a run per lane, and the pages of the 32 after those: look-ups are never waited for in the loop
    const int first = seg.k0 * GROUP;
    const int n = max(0, min(seg.k0 + seg.n, (x.hi + GROUP - 1) / GROUP) - seg.k0);  // steps
    const int* const row = c.table + (long long)s.slot * c.table_stride;
    constexpr int UNSEEN = -1, MISSING = -2;
    auto lookup = [&](int r) {
      const int j = first + (r << a.run_shift);
      if (r >= n << runs_shift || j >= x.hi || j + (1 << a.run_shift) <= x.lo) return UNSEEN;  // no row sees it
      const int p = row[j >> a.shift];
      if ((unsigned)p < (unsigned)c.num_pages) return p;
      raise(c.status, FAKV_BAD_PAGE);
      return MISSING;
    };
    int page = UNSEEN, page_next = lookup(lane);
    const uint8_t *codes = a.qc.K, *params_of = a.qc.K;  // of the lane's run in K
    ptx::fence_async_shared();  // what was written to the ring by threads comes before the copies
    __syncwarp();

    // ---- copies of step i's K and V, a run by each lane whose run is one of the step's: the keys that no row
    // sees stay what they are, those of a missing page are zeros. `at`: the step's place in the ring
    auto load = [&](int i, uint32_t at, uint64_t* bar) {
      if (i >= n) return;
      if ((i & (31 >> runs_shift)) == 0) {
        page = page_next;
        const int r = (i << runs_shift) + lane, t = (first + (r << a.run_shift)) & (c.page_size - 1);
        const uint8_t* const block = a.qc.K + seg.head * a.qc.head + max(page, 0) * a.qc.page;
        codes = block + t * chunks * 16;
        params_of = block + a.qc.params + t * NG * 4;
        page_next = lookup(r + 32);
      }
      if ((lane >> runs_shift) == (i & (31 >> runs_shift))) {
        const int r = lane & ((1 << runs_shift) - 1);
        const uint32_t to = at + r * (CH * 16 << a.run_shift), to_p = at + C::CODES + r * (NG * 4 << a.run_shift);
        if (page >= 0) {
          ptx::mbar_arrive_expect_tx(bar, 2 * (run_codes + run_params));
          bulk_load(to, codes, run_codes, bar);
          bulk_load(to_p, params_of, run_params, bar);
          bulk_load(to + C::SLOT, codes + v_minus_k, run_codes, bar);
          bulk_load(to_p + C::SLOT, params_of + v_minus_k, run_params, bar);
        } else {
          if (page == MISSING) {
            for (int v = 0; v < 2; ++v) {
              for (uint32_t k = 0; k < run_codes; k += 16) ptx::st_shared_v4(to + v * C::SLOT + k, 0, 0, 0, 0);
              for (uint32_t k = 0; k < run_params; k += 16) ptx::st_shared_v4(to_p + v * C::SLOT + k, 0, 0, 0, 0);
            }
            ptx::fence_async_shared();
          }
          ptx::mbar_arrive(bar);
        }
      }
    };

    // ---- q: fragments of its rows (zeros behind the item's rows and the tensor's columns), each row
    // times a power of two; of rows 8 nt + 2 quad + e the sums over each group, and what makes logits (log2) of
    // their scores
    uint4 qr[C::Q_REGS ? KS / 2 : 1];
    float2 qs[NTR][NG], ql[NTR];
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) {
      const int r = nt * 8 + oct;
      const int rho = x.rho0 + min(r, x.rows - 1), token = g.rep.of(rho);
      const E* const from = static_cast<const E*>(a.q) + (s.row0 + token) * a.q_token +
                            (seg.head * g.rep.d + rho - token * g.rep.d) * a.q_head;
      float y[KS / 2][8];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i)  // two k16 steps: 4 bits: 8 columns of block i; 8 bits: 4 of chunks 2 i and 2 i + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // four columns each
          const int col = BITS == 4 ? i * 32 + quad * 8 + e * 4 : (2 * i + e) * 16 + quad * 4;
          float* const to = &y[i][4 * e];
          to[0] = to[1] = to[2] = to[3] = 0.f;
          if (r < x.rows && col < c.D) {
            if constexpr (C::F32) {
              const float4 v = *reinterpret_cast<const float4*>(from + col);
              to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(from + col);
              to[0] = __uint_as_float(v.x << 16); to[1] = __uint_as_float(v.x & 0xffff0000u);
              to[2] = __uint_as_float(v.y << 16); to[3] = __uint_as_float(v.y & 0xffff0000u);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(to[k]));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(q_exponent(top), -100), 127);
      const float down = q_pow2(14 - e), up = fmaxf(a.sl2 * q_pow2(e - 14), FLT_MIN);  // (a masked score is -infinity times it)
      // (infinity in a row makes all that it sees NaN, whatever the codes)
      float sum[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) sum[i] = top < INFINITY ? 0.f : __int_as_float(0x7fffffff);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        // of the code pairs: 4 bits (0, 4), (1, 5), (2, 6), (3, 7); 8 bits (0, 1), (2, 3) of each chunk
        uint32_t f[2][4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int c0 = BITS == 4 ? z : 2 * z, c1 = BITS == 4 ? z + 4 : 2 * z + 1;
          const float factor = q_factor<BITS>(CENTRED ? 1 : z);
          float2 v = make_float2(y[i][c0] * (down / factor), y[i][c1] * (down / factor));
          sum[NG > 1 ? i / 2 : 0] += (v.x + v.y) * factor;
          f[0][z] = half2_of(v.x, v.y, &v);
          f[1][z] = half2_of(v.x, v.y);
        }
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          if constexpr (C::Q_REGS) qr[i] = make_uint4(f[0][0], f[0][1], f[0][2], f[0][3]);
          else ptx::st_shared_v4(sq + ((nt * TERMS + t) * (KS / 2) + i) * 512 + lane * 16, f[t][0], f[t][1], f[t][2], f[t][3]);
        }
      }
      // (a row's own lanes' value, to the lanes that have the row's scores)
      auto of_row = [&](float v) { return make_float2(__shfl_sync(0xffffffffu, v, 8 * quad), __shfl_sync(0xffffffffu, v, 8 * quad + 4)); };
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        qs[nt][i] = of_row(sum[i]);
      }
      ql[nt] = of_row(up);
    }
    __syncwarp();

    // rows 8 nt + 2 quad + e; o: of each tile, two adjacent columns of the lane's
    float o[CH][VT][NTR][4];
    float2 m[NTR], l[NTR], oz[NTR][NG];
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) {
      m[nt] = make_float2(-FLT_MAX, -FLT_MAX);
      l[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NG; ++i) oz[nt][i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < CH; ++w)
#pragma unroll
        for (int t = 0; t < VT; ++t) o[w][t][nt][0] = o[w][t][nt][1] = o[w][t][nt][2] = o[w][t][nt][3] = 0.f;
    }
    // keys that every row sees need no mask
    int in_lo, in_hi;
    {
      const int pa = s.len - s.n + g.rep.of(x.rho0), pb = s.len - s.n + g.rep.of(x.rho0 + x.rows - 1);
      in_hi = g.causal ? min(pa, s.len - 1) : s.len - 1;
      in_lo = g.window > 0 ? pb - g.window + 1 : 0;
    }

    // Steps of GROUP keys, whose place is filled again as soon as it is read, NP steps ahead.
    // V's scales that a row has seen, times its lift, are at most 2^6 (before the first one: any is above it)
    float2 lift[NTR];
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) lift[nt] = make_float2(NO_LIFT, NO_LIFT);
#pragma unroll 1
    for (int k = 0; k < min(n, NP); ++k) {
      const int at = ring + k < NP ? ring + k : ring + k - NP;
      load(k, sq + C::Q_BYTES + at * 2 * C::SLOT, &bars[warp][at]);
    }
    int i = 0;
#pragma unroll 1
    for (; i < n; ++i) {
      const int j0 = first + i * GROUP;
      const bool edge = j0 < in_lo || j0 + GROUP - 1 > in_hi;
      const uint32_t use = C::Q_BYTES + ring * 2 * C::SLOT;  // the step's place in the warp's shared memory
      uint64_t* const bar = &bars[warp][ring];
      float2 sc[KT][NTR][2];  // scores, then probabilities: keys 16 kt + 8 z + oct, rows 8 nt + 2 quad, + 1
      if (!(ok = wait(bar))) break;
      const uint8_t* const slot_v = mine + use + C::SLOT;
      {
        const uint8_t* const slot = mine + use;
        // -------- scores
        // (chunks that the cache does not have: whatever lies in the slot, finite codes, times q's zeros)
        float acc[NG][KT][NTR][4];
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[k][kt][nt][e] = 0.f;
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const int k = NG == 1 ? 0 : BITS == 4 ? w / 2 : w / 4;  // the chunk's group
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            uint32_t word[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              word[e] = *reinterpret_cast<const uint32_t*>(slot + ((kt * 2 + e) * CH + w) * 128 + lane * 4);
            auto product = [&](auto pair, uint32_t b0, uint32_t b1, int nt) {  // code pairs `pair` and + 1
              constexpr int P = decltype(pair)::value;
              uint32_t f[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                f[e] = CENTRED ? q_centred<BITS, 1>(q_raise16<BITS, P>(word[e], a.raised)) : q_small<BITS, P>(word[e]);
                f[2 + e] = CENTRED ? q_centred<BITS, 1>(q_raise16<BITS, P + 1>(word[e], a.raised)) : q_small<BITS, P + 1>(word[e]);
              }
              mma_f16(acc[k][kt][nt], f, b0, b1);
            };
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int t = TERMS - 1; t >= 0; --t) {
                const int step = BITS == 4 ? w : w / 2;
                uint4 v;
                if constexpr (C::Q_REGS) v = qr[step];
                else v = *reinterpret_cast<const uint4*>(mine + ((nt * TERMS + t) * (KS / 2) + step) * 512 + lane * 16);
                if constexpr (BITS == 4) {
                  product(std::integral_constant<int, 0>(), v.x, v.y, nt);
                  product(std::integral_constant<int, 2>(), v.z, v.w, nt);
                } else {
                  product(std::integral_constant<int, 0>(), w & 1 ? v.z : v.x, w & 1 ? v.w : v.y, nt);
                }
              }
          }
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t p[NG];
            params(slot, kt, z, p);
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt) {
              float2 v = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < NG; ++k) {
                const float ps = CENTRED ? q_scale(p[k]) : q_scale24(p[k]), pz = CENTRED ? fmaf(ps, CENTRE, q_offset(p[k])) : q_offset(p[k]);
                v.x = k == 0 ? pz * qs[nt][k].x : fmaf(pz, qs[nt][k].x, v.x);
                v.y = k == 0 ? pz * qs[nt][k].y : fmaf(pz, qs[nt][k].y, v.y);
                v.x = fmaf(ps, acc[k][kt][nt][2 * z], v.x);
                v.y = fmaf(ps, acc[k][kt][nt][2 * z + 1], v.y);
              }
              sc[kt][nt][z] = v;
            }
          }
        // (what a row does not see has no part in it: scores -infinity; V's scales, which may be those of no token, passed over)
        float2 most[NTR];  // the largest of V's scales among the lane's keys that the row sees (NaN is passed over)
        {
          float top[KT][2];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t p[NG];
              params(slot_v, kt, z, p);
              top[kt][z] = NG == 1 ? q_scale(p[0]) : fmaxf(q_scale(p[0]), q_scale(p[NG - 1]));
            }
          if (edge) {
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // row 8 nt + 2 quad + e sees keys [lo, hi]
                const int p = s.len - s.n + g.rep.of(x.rho0 + min(nt * 8 + quad * 2 + e, x.rows - 1));
                const int hi = g.causal ? min(p, s.len - 1) : s.len - 1;
                const int lo = g.window > 0 ? p - g.window + 1 : 0;
                float all = 0.f;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    const int key = j0 + kt * 16 + z * 8 + oct;
                    if (key < lo || key > hi) (e ? sc[kt][nt][z].y : sc[kt][nt][z].x) = -INFINITY;
                    else all = fmaxf(all, top[kt][z]);
                  }
                (e ? most[nt].y : most[nt].x) = all;
              }
          } else {
            float all = 0.f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) all = ptx::max3(all, top[kt][0], top[kt][1]);
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt) most[nt] = make_float2(all, all);
          }
        }
        // -------- probabilities; m, and the power of two on V's scales, where they have to move
        float2 mx[NTR];
        float2 by[NTR];  // (ql, or 1 where the scores have been multiplied with it)
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NTR; ++nt) {
          mx[nt] = make_float2(fmaxf(sc[0][nt][0].x, sc[0][nt][1].x), fmaxf(sc[0][nt][0].y, sc[0][nt][1].y));
#pragma unroll
          for (int kt = 1; kt < KT; ++kt)
            mx[nt] = make_float2(ptx::max3(mx[nt].x, sc[kt][nt][0].x, sc[kt][nt][1].x), ptx::max3(mx[nt].y, sc[kt][nt][0].y, sc[kt][nt][1].y));
          mx[nt] = make_float2(mx[nt].x * ql[nt].x, mx[nt].y * ql[nt].y);
          grow |= mx[nt].x > m[nt].x + RESCALE_THRESHOLD || mx[nt].y > m[nt].y + RESCALE_THRESHOLD;
          grow |= most[nt].x * lift[nt].x > 64.f || most[nt].y * lift[nt].y > 64.f;
          grow |= fabsf(m[nt].x) > Q_LARGE || fabsf(m[nt].y) > Q_LARGE;
          by[nt] = ql[nt];
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NTR; ++nt) {
            float2 f, fv;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              auto over_keys = [](float v) {
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              };
              // (a row by itself, and by the keys that it sees: not as its neighbours' scores fall, or a key's V that is theirs)
              const float v = over_keys(e ? mx[nt].y : mx[nt].x), top = over_keys(e ? most[nt].y : most[nt].x);
              float& had = e ? lift[nt].y : lift[nt].x;
              float to = had;
              if (top * had > 64.f) to = q_pow2(5 - min(max(q_exponent(top), -100), 126));  // (twice as large may come before the next move)
              (e ? fv.y : fv.x) = to / had;
              had = to;
              float& was = e ? m[nt].y : m[nt].x;
              const float mn = v > was + RESCALE_THRESHOLD ? v : was;
              (e ? f.y : f.x) = ptx::ex2(was - mn);
              was = mn;
              if (fabsf(mn) > Q_LARGE) {
                const float l = e ? ql[nt].y : ql[nt].x;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                  for (int z = 0; z < 2; ++z) (e ? sc[kt][nt][z].y : sc[kt][nt][z].x) *= l;
                (e ? by[nt].y : by[nt].x) = 1.f;
              }
            }
            l[nt] = ptx::mul2(l[nt], f);
#pragma unroll
            for (int k = 0; k < NG; ++k) oz[nt][k] = ptx::mul2(oz[nt][k], f);
            f = ptx::mul2(f, fv);
#pragma unroll
            for (int w = 0; w < CH; ++w)
#pragma unroll
              for (int t = 0; t < VT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[w][t][nt][e] *= e & 1 ? f.y : f.x;
          }
          __syncwarp();  // (rows move by themselves: together again for the products)
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float2 v = ptx::fma2(sc[kt][nt][z], by[nt], make_float2(-m[nt].x, -m[nt].y));
              sc[kt][nt][z] = make_float2(ptx::ex2(v.x), ptx::ex2(v.y));
              l[nt] = ptx::add2(l[nt], sc[kt][nt][z]);
            }
        // -------- O^T += V^T (s P)^T, and the offsets' sums
        uint32_t pf[KT][NG][NTR][PT][2];  // terms of s P; keys low, high
        auto weigh = [&](auto masked) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int k = 0; k < NG; ++k) {
                uint32_t pv[NG];
                params(slot_v, kt, z, pv);
                const float ps = q_scale(pv[k]), pz = fmaf(ps, CENTRE, q_offset(pv[k]));
#pragma unroll
                for (int nt = 0; nt < NTR; ++nt) {
                  const float2 p = sc[kt][nt][z], pl = ptx::mul2(make_float2(ps, ps), lift[nt]);
                  float2 sp;
                  if constexpr (decltype(masked)::value) {  // a key that a row does not see may be anything
                    sp = make_float2(p.x == 0.f ? 0.f : p.x * pl.x, p.y == 0.f ? 0.f : p.y * pl.y);
                    oz[nt][k].x += p.x == 0.f ? 0.f : p.x * pz;
                    oz[nt][k].y += p.y == 0.f ? 0.f : p.y * pz;
                  } else {
                    sp = ptx::mul2(p, pl);
                    oz[nt][k].x = fmaf(p.x, pz, oz[nt][k].x);
                    oz[nt][k].y = fmaf(p.y, pz, oz[nt][k].y);
                  }
#pragma unroll
                  for (int t = 0; t < PT; ++t) pf[kt][k][nt][t][z] = transpose8(half2_of(sp.x, sp.y, &sp));
                }
              }
        };
        if (edge) weigh(std::true_type());
        else weigh(std::false_type());
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
          for (int w = 0; w < CH; ++w) {
            const int k = NG == 1 ? 0 : BITS == 4 ? w / 2 : w / 4;  // the chunk's group
            uint32_t word[2];  // of keys low, high: codes of two keys side by side
#pragma unroll
            for (int z = 0; z < 2; ++z)
              word[z] = *reinterpret_cast<const uint32_t*>(slot_v + ((kt * 2 + z) * CH + w) * 128 + quad * 32 + oct * 4);
            auto tile = [&](auto jj) {
              constexpr int t = decltype(jj)::value, P = 2 * t;
              const uint32_t va[4] = {q_centred<BITS, P>(q_raise<BITS, P>(word[0], a.raised)), q_centred<BITS, P + 1>(q_raise<BITS, P + 1>(word[0], a.raised)),
                                      q_centred<BITS, P>(q_raise<BITS, P>(word[1], a.raised)), q_centred<BITS, P + 1>(q_raise<BITS, P + 1>(word[1], a.raised))};
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt) {
                if constexpr (PT == 1) {
                  mma_f16(o[w][t][nt], va, pf[kt][k][nt][0][0], pf[kt][k][nt][0][1]);
                } else {  // a sum per 16 keys, added to O in fp32: O itself is not cut off at every product
                  float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                  for (int b = PT - 1; b >= 0; --b) mma_f16(add, va, pf[kt][k][nt][b][0], pf[kt][k][nt][b][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[w][t][nt][e] += add[e];
                }
              }
            };
            tile(std::integral_constant<int, 0>());
            if constexpr (BITS == 4) tile(std::integral_constant<int, 1>());
          }
        }
      }
      __syncwarp();  // the codes are read
      load(i + NP, sq + use, bar);
      if (++ring == NP) {
        ring = 0;
        parity ^= 1;
      }
    }
    if (!ok) {
      // a wait ran out: nothing more is asked for, and what is in flight is given time to land
      for (int k = i; k < min(n, i + NP); ++k) {
        const int at = ring + k - i;
        const uint64_t t0 = ptx::globaltimer();
        while (!ptx::mbar_try_wait(&bars[warp][at % NP], parity ^ (at / NP & 1)) && ptx::globaltimer() - t0 < WAIT_LIMIT_NS / 16) {}
      }
      held = false;
      break;
    }

    // ---- this warp's sums into its shared memory
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        auto over_keys = [](float v) {
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          return v + __shfl_xor_sync(0xffffffffu, v, 16);
        };
        const float v = over_keys(e ? l[nt].y : l[nt].x);
        float z[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) z[i] = over_keys(e ? oz[nt][i].y : oz[nt][i].x);
        const int r = nt * 8 + quad * 2 + e;
        if (oct == 0) ends_sh.ml[warp][r] = make_float2(e ? m[nt].y : m[nt].x, v);
        float* const to = reinterpret_cast<float*>(mine) + r * C::OS + oct * 2 * VT;
        const float by = 1.f / (e ? lift[nt].y : lift[nt].x);
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const float zw = z[NG == 1 ? 0 : BITS == 4 ? w / 2 : w / 4];
#pragma unroll
          for (int t = 0; t < VT; ++t)
            *reinterpret_cast<float2*>(to + w * 16 * VT + 2 * t) =
                make_float2(fmaf(o[w][t][nt][e], by, zw), fmaf(o[w][t][nt][e + 2], by / q_factor<BITS>(1), zw));
        }
      }
    fin = {s.row0, x.rho0, x.rows, seg.head, walk.p.ender,
           (seg.starts ? PART_STARTS : 0) | (seg.ends ? PART_ENDS : 0), 2 * worker + seg.slot};
    __syncwarp();
    held = seg.slot == 0 && walk.done() && !(seg.starts && seg.ends);
    if (!held) {
      finish<C, D>(a, fin, smem, ends_sh.ml, warp, warp, lane, 32);
      __syncwarp();
    }
  }

  finish_held<C, D>(a, fin, held, walk.moved, smem, ends_sh);
}

template <typename E, bool OUT_BF, int BITS, int D, int NG, int NTR>
fa_status run(QRowsArgs& a, cudaStream_t s) {
  using C = QRowsCfg<E, OUT_BF, BITS, D, NG, NTR>;
  auto* kernel = qattend_rows_kernel<E, OUT_BF, BITS, D, NG, NTR>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return failed();
  const int ctas = host::sm_count() * C::CTAS_PER_SM;
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas * WARPS, C::R, D), s) != cudaSuccess) return failed();
  a.part = partials_at(w, ctas * WARPS, C::R, D);
  // (fewer chunks than the slots have room for: their octets are not one after another there)
  a.run_shift = a.qc.chunks == C::CH ? std::min(a.shift, log2_of(C::GROUP)) : 3;
  a.g.R = C::R;
  a.g.u_shift = log2_of(C::GROUP);
  a.g.start = 4;  // steps: looking up an item's first pages and rows takes about as long
  a.g.snap = 4;
  fa_status st;
  {
    host::KernelTimer t("qattend_rows", s);
    st = launch(kernel, ctas, NTHREADS, C::SMEM, s, a);
  }
  if (st == FA_OK) {
    const JoinArgs j = {a.part, a.O, a.LSE, ctas, WARPS, C::R, D, a.H, a.c.D, a.out_bf16, a.g.rep};
    st = launch_join(j, s);
  }
  if (host::scratch_free(w, s) != cudaSuccess) st = failed();
  return st;
}

template <typename E, bool OUT_BF, int BITS, int NTR>
fa_status pick(QRowsArgs& a, cudaStream_t s) {
  if (a.c.D <= 64) return run<E, OUT_BF, BITS, 64, 1, NTR>(a, s);
  return a.qc.groups == 1 ? run<E, OUT_BF, BITS, 128, 1, NTR>(a, s) : run<E, OUT_BF, BITS, 128, 2, NTR>(a, s);
}
template <typename E, bool OUT_BF>
fa_status pick(QRowsArgs& a, long long rows, cudaStream_t s) {
  if (a.qc.bits == 4) return rows <= 8 ? pick<E, OUT_BF, 4, 1>(a, s) : pick<E, OUT_BF, 4, 2>(a, s);
  return rows <= 8 ? pick<E, OUT_BF, 8, 1>(a, s) : pick<E, OUT_BF, 8, 2>(a, s);
}

}  // namespace

fa_status launch_qattend_rows(const void* q, void* O, float* LSE, const int* cu, const int* slots, const QCache& qc,
                              const fakv_tokens& p, cudaStream_t s) {
  QRowsArgs a = {};
  const fakv_cache& c = qc.c;
  a.c = c;
  a.qc = qc;
  a.q = q;
  a.O = O;
  a.LSE = LSE;
  a.cu = cu;
  a.slots = slots;
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.shift = log2_of(c.page_size);
  a.q_token = p.q_token;
  a.q_head = p.q_head;
  const int rep = p.H / c.HKV;
  a.g.rep = div_by(rep);
  a.g.causal = p.causal;
  a.g.window = p.window;
  a.sl2 = p.scale * LOG2E;
  a.raised = Q_RAISED;
  a.out_bf16 = p.out_dtype == FA_BF16;
  // Items of 8 or 16 rows: what a sequence's rows fit on average
  const long long rows = ((long long)p.T * rep + p.B - 1) / p.B;
  if (c.dtype == FA_BF16) return a.out_bf16 ? pick<__nv_bfloat16, true>(a, rows, s) : pick<__nv_bfloat16, false>(a, rows, s);
  return pick<float, false>(a, rows, s);
}

unsigned int read_and_clear_kvq_status(cudaError_t* err) {
  unsigned int v = 0, zero = 0;
  *err = cudaMemcpyFromSymbol(&v, g_kvq_status, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_kvq_status, &zero, sizeof(zero));
  return v;
}

}  // namespace kv
}  // namespace fa
