// kv_rows.cu -- attention over the paged cache for few rows per sequence (decoding), and
// for fp32 caches: K and V streamed once, mma.sync.
//
// Few rows read many keys: 4 D flops per row against 4 D bytes (bf16) per key, so up to a
// few dozen rows the work is bound by HBM. A warp is a worker (kv_sched.cuh): it walks its
// part of the line on its own, in groups of keys (4 KB of K, 4 KB of V) that it copies with
// cp.async (any page size and stride, no copy descriptor to build on the host) into a ring
// of its own; K and V slots are refilled as soon as each is read. Where one warp changes
// items, the SM's others (eleven, or seven) keep the memory busy, and the loop has no CTA
// barrier. (With a CTA per item, 64 sequences of 512 tokens on average took 45 us instead of
// 35, 20 being the floor: every item drained and refilled the CTA's whole pipeline.) Only
// where all warps of a CTA end up with one and the same item do they put their results
// together in shared memory, so that a long sequence leaves a part per CTA to join.
//
// Measured (32 query heads on 8 kv heads of 128, one new token each, pages of 16): 64 sequences
// of up to 16384 tokens 337 to 350 us, 2.15 GB at 6.1 to 6.4 TB/s, 0.91 to 0.94 of the measured
// copy rate (a sixteenth of it is the join); 64 of up to 1024 36 us (floor 20), 16 of up to 8192
// 58 (44); one sequence of 16 tokens 8.3 us and of 1021 9.7 us, which is
// latency: 1.6 us from the launch to the cuts, 1.6 us to the first keys asked for, 0.5 us to
// have them, 4 us the join. fp32: 64 sequences of up to 8192 346 us, 2.15 GB; 12 of up to 5 new
// tokens, window 1024, heads of 64: 16.8 us with their 48 MB in L2 and 20.9 without; its three
// products per GEMM and their splits are what bounds it.
//
//   scores  S^T = K Q^T: the 16 rows of an mma tile are keys, its 8 columns rows of q, so
//           that eight rows (a decoding step) cost eight rows. bf16 m16n8k16, fp32 sums.
//           fp32 caches: x = hi + lo with tf32 terms, hi hi + hi lo + lo hi (m16n8k8).
//   softmax online in the exp2 domain; m moves only when a score would exceed it by more than
//           8 (the sums stay exact: every exponential of an item is taken against the
//           same m as its O), so a step asks with one vote and reduces nothing.
//   O^T += V^T P^T  bf16: P = hi + lo, two bf16 terms, so that P's rounding (2^-8) does not
//           add to the output's: the second product is free under the memory time.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include "kv_sched.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int WARPS = 4;
constexpr int NTHREADS = 32 * WARPS;

struct RowsArgs {
  fakv_cache c;
  const void* q;
  void* O;
  float* LSE;
  const int* cu;
  const int* slots;
  int B, T, H, plane, shift;
  long long q_token, q_head;
  Geo g;
  float sl2;  // scale * log2(e)
  int out_bf16;
  Partials part;
};

template <typename E, int D, int NTR>
struct RowsCfg {
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int R = 8 * NTR;               // rows of an item
  static constexpr int RB = D * (int)sizeof(E);   // bytes of a K / V / Q row
  static constexpr int CH = RB / 16;              // 16-byte chunks of it
  static constexpr int GROUP = 4096 / RB > 16 ? 4096 / RB : 16;  // keys of a group
  static constexpr int KT = GROUP / 16;           // 16-key tiles of it
  static constexpr int SLOT = GROUP * RB;         // K (or V) of a group
  static constexpr int Q_BYTES = R * RB;
  // Bytes on their way per SM: 12 warps x 4 slots, or 8 x 6, of 4 KB hold 192 KB, a latency of
  // 2 us or more at the SM's share of HBM; three CTAs where the registers allow them,
  // because more warps hide a change of items better.
  static constexpr int WANT = NTR == 1 && RB < 512 ? 3 : 2;
  static constexpr int ROOM = WANT == 3 ? 18432 : NTR <= 2 ? 28672 : 28160;
  static constexpr bool FITS = ROOM - Q_BYTES >= 2 * SLOT;
  static constexpr int CTAS_PER_SM = FITS ? WANT : 1;
  static constexpr int NS = ((FITS ? ROOM : 56320) - Q_BYTES) / SLOT;
  static constexpr int WARP_BYTES = NS * SLOT + Q_BYTES;
  static constexpr int SMEM = WARPS * WARP_BYTES;
  static constexpr int OS = D + 4;                // floats of a row of O in shared memory (bank spread)
  static constexpr bool Q_REGS = NTR == 1 && (!F32 || D == 64);  // q's fragments stay in registers
  static_assert(NS >= 2 && WARP_BYTES >= R * OS * 4, "a warp's ring also holds its O at the end");
  static_assert(SMEM >= 4 * 16385, "the plan's scratch");
  static constexpr int STATIC = (int)sizeof(PlanShared<NTHREADS, WARPS>) + WARPS * (R * 8 + 20);
  static_assert(CTAS_PER_SM * (SMEM + (STATIC + 1023) / 1024 * 1024 + 1024) <= 228 * 1024, "shared memory of the CTAs of an SM");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi the value rounded to tf32's 11 significant bits (half of the 13 low bits'
// step added before they go), lo the rest, of which the tensor core cuts off the low bits.
// Rounded, hi leaves a lo of either sign, so that lo's cut and the missing lo lo products
// do not add up (with hi cut off as well, O was 2.7e-6 off instead of 0.6e-6).
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
  hi = (x + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// chunk of a row in shared memory (16-byte chunks, spread so that the eight rows of an
// ldmatrix, or the eight (key, column) chunks of a scalar fp32 V read, fall in different banks)
template <int RB>
__device__ __forceinline__ uint32_t at_rows(int row, int chunk) {
  return (uint32_t)(row * RB + ((chunk ^ (row & 7)) << 4));
}
template <int RB>
__device__ __forceinline__ uint32_t at_v32(int row, int chunk) {
  return (uint32_t)(row * RB + ((chunk ^ ((row & 3) << 1)) << 4));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // of an 8 x 8 matrix of 16-bit values
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Sums of exponentials taken against the maximum M. L = 0: no key seen. (Tested for 0, not for
// its sign: NaN sums, from a row of q or a page, are sums, and reach O and LSE however the item was cut.)
struct Sum {
  float M, L;
  float4 acc;
  __device__ __forceinline__ void add(float m, float l, const float4& v) {
    const float mn = fmaxf(M, m);
    const float fo = ptx::ex2(M - mn), fn = ptx::ex2(m - mn);
    M = mn;
    L = L * fo + l * fn;
    acc.x = acc.x * fo + v.x * fn;
    acc.y = acc.y * fo + v.y * fn;
    acc.z = acc.z * fo + v.z * fn;
    acc.w = acc.w * fo + v.w * fn;
  }
  // columns col .. col + 3 of row `at` of O [.][cols], and its LSE
  __device__ __forceinline__ void write(void* O, float* LSE, size_t at, int col, int cols, bool bf16) const {
    const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
    if (col == 0) LSE[at] = L == 0.f ? -INFINITY : (M + __log2f(L)) * LN2;
    if (col >= cols) return;
    if (bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(O) + at * cols + col) =
          make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(O) + at * cols + col) =
          make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
};

// An item's (or its part's) result from the sums of warps w0 .. w1 of the CTA, each in its own
// shared memory: O [R][OS] not normalised, m and l in ml. By `threads` threads of which the
// caller is number i. flags: PART_STARTS, PART_ENDS (both: the whole item), PART_JOINED.
struct Finish {
  int row0, rho0, rows, head, ender, flags, slot;
};
template <typename C, int D>
__device__ __forceinline__ void finish(const RowsArgs& a, const Finish& f, const uint8_t* smem,
                                    const float2 (*ml)[C::R], int w0, int w1, int i, int threads) {
  const bool whole = (f.flags & PART_STARTS) && (f.flags & PART_ENDS);
  constexpr int COLS = D / 4;  // threads of a row
  const int col = i % COLS * 4;
  for (int r = i / COLS; r < f.rows; r += threads / COLS) {
    auto of = [&](int w) {
      return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * C::WARP_BYTES) + r * C::OS + col);
    };
    Sum x = {ml[w0][r].x, ml[w0][r].y, of(w0)};
#pragma unroll 1
    for (int w = w0 + 1; w <= w1; ++w) x.add(ml[w][r].x, ml[w][r].y, of(w));
    if (whole) {
      const int rho = f.rho0 + r, token = a.g.rep.of(rho);
      x.write(a.O, a.LSE, (size_t)(f.row0 + token) * a.H + f.head * a.g.rep.d + rho - token * a.g.rep.d, col, a.c.D,
              a.out_bf16);
    } else {
      *reinterpret_cast<float4*>(a.part.O + ((size_t)f.slot * C::R + r) * D + col) = x.acc;
      if (col == 0) a.part.ml[(size_t)f.slot * C::R + r] = make_float2(x.M, x.L);
    }
  }
  if (!whole && i == 0)
    a.part.left[f.slot] = {f.flags, f.row0, f.rho0, f.rows, f.head, f.ender, {0, 0}};
}

template <typename E, int D, int NTR>
__global__ void __launch_bounds__(NTHREADS, RowsCfg<E, D, NTR>::CTAS_PER_SM)
    attend_rows_kernel(const __grid_constant__ RowsArgs a) {
  using C = RowsCfg<E, D, NTR>;
  constexpr int RB = C::RB, CH = C::CH, R = C::R, NS = C::NS, GROUP = C::GROUP, KT = C::KT;
  constexpr int EPC = 16 / (int)sizeof(E);  // elements of a chunk
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ PlanShared<NTHREADS, WARPS> plan;
  __shared__ float2 ml_sh[WARPS][R];
  __shared__ int4 item_sh[WARPS];  // b, tile, head, and 1: held, 2: no part, 0: neither
  __shared__ int ends_sh[WARPS];   // a held item's PART_STARTS, PART_ENDS
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, oct = lane >> 2;  // mma fragments: columns 2 quad, 2 quad + 1; row oct
  const int mat = lane >> 3, mr = lane & 7;    // ldmatrix: matrix, row
  const fakv_cache& c = a.c;
  const Geo& g = a.g;
  Seq seq;
  const Part part = find_part<NTHREADS, WARPS>(g, c, a.cu, a.slots, a.B, a.T, reinterpret_cast<int*>(smem), plan, seq);
  Walk walk(part, seq);
  const int worker = blockIdx.x * WARPS + warp;
  if (lane < 2) a.part.left[2 * worker + lane].flags = 0;
  if (lane == 0) item_sh[warp] = make_int4(walk.p.b, walk.p.tile, walk.p.head, 2);
  uint8_t* const mine = smem + warp * C::WARP_BYTES;
  const uint32_t sq = ptx::smem_u32(mine);
  const uint32_t ring = sq + C::Q_BYTES;
  const int dv_chunks = c.D / EPC;
  const E* const Kp = static_cast<const E*>(c.K) + a.plane * c.plane_stride;
  const E* const Vp = static_cast<const E*>(c.V) + a.plane * c.plane_stride;
  Seg seg = {};
  Finish fin;
  bool held = false;  // the worker's only item, not done whole: its result waits for the others'

  while (walk.next(g, c, a.cu, a.slots, a.T, seg)) {
    const Seq& s = seg.s;
    const Tile& x = seg.x;

    // ---- pages of the next 32 octets of keys, an octet per lane, and of the 32 after those:
    // look-ups are never waited for in the loop
    const int first = seg.k0 * GROUP;
    const int n = max(0, min(seg.k0 + seg.n, (x.hi + GROUP - 1) / GROUP) - seg.k0);  // groups
    const int* const row = c.table + (long long)s.slot * c.table_stride;
    auto lookup = [&](int octet) {
      const int j = first + octet * 8;
      if (octet >= n * (GROUP / 8) || j >= x.hi || j + 8 <= x.lo) return -1;  // no row sees it
      const int p = row[j >> a.shift];
      if ((unsigned)p < (unsigned)c.num_pages) return p;
      raise(c.status, FAKV_BAD_PAGE);
      return -1;
    };
    int page = -1, page_next = lookup(lane);

    // ---- q rows (zeros behind the item's rows and the tensor's columns)
#pragma unroll 1
    for (int i = lane; i < R * CH; i += 32) {
      const int r = i / CH, ch = i % CH;
      const int rho = x.rho0 + r, token = g.rep.of(rho);
      const bool in = r < x.rows && ch < dv_chunks;
      const E* src = static_cast<const E*>(a.q);
      if (in) src += (s.row0 + token) * a.q_token + (seg.head * g.rep.d + rho - token * g.rep.d) * a.q_head + ch * EPC;
      cp16(sq + at_rows<RB>(r, ch), src, in);
    }

    // ---- copies of half-step j: K (j even) or V of group j / 2, octet by octet, each in a page
    long long base[GROUP / 8];  // of the group's octets (-1: zeros)
    uint32_t fill = ring;
    auto load = [&](int j) {
      if (j < 2 * n) {
        const bool is_v = j & 1;
        const E* const src = (is_v ? Vp : Kp) + seg.head * c.head_stride;
#pragma unroll
        for (int k = 0; k < GROUP / 8; ++k) {
          const int octet = (j >> 1) * (GROUP / 8) + k;
          const int key = first + octet * 8;
          if (!is_v) {
            if ((octet & 31) == 0) {
              page = page_next;
              page_next = lookup(octet + 32 + lane);
            }
            const int p = __shfl_sync(0xffffffffu, page, octet & 31);
            base[k] = p < 0 ? -1 : p * c.page_stride + (key & (c.page_size - 1)) * c.token_stride;
          }
#pragma unroll
          for (int z = 0; z < 8 * CH / 32; ++z) {
            const int r = (z * 32 + lane) / CH, ch = (z * 32 + lane) % CH;
            // what no row sees is not read: it may hold anything
            const bool in = base[k] >= 0 && key + r >= x.lo && key + r < x.hi && ch < dv_chunks;
            const E* const p = in ? src + base[k] + r * c.token_stride + ch * EPC : src;
            cp16(fill + (C::F32 && is_v ? at_v32<RB>(8 * k + r, ch) : at_rows<RB>(8 * k + r, ch)), p, in);
          }
        }
        fill = fill + C::SLOT == ring + NS * C::SLOT ? ring : fill + C::SLOT;
      }
      cp_commit();
    };

    float m[NTR][2], l[NTR][2], o[D / 16][NTR][4];  // rows 8 nt + 2 quad + e
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) {
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[d][nt][0] = o[d][nt][1] = o[d][nt][2] = o[d][nt][3] = 0.f;
    }
    // keys that every row sees need no mask
    int in_lo, in_hi;
    {
      const int pa = s.len - s.n + g.rep.of(x.rho0), pb = s.len - s.n + g.rep.of(x.rho0 + x.rows - 1);
      in_hi = g.causal ? min(pa, s.len - 1) : s.len - 1;
      in_lo = g.window > 0 ? pb - g.window + 1 : 0;
    }

    // Half-steps K_0, V_0, K_1, ...: a slot is filled again as soon as it is read, NS half-steps
    // ahead. The first NS rounds only load: one copy of the loading code, as every instruction
    // that is new costs its fetch.
    uint32_t use = ring;
    float sc[KT][NTR][4];  // scores, then probabilities: keys 16 kt + oct (+ 8), rows 8 nt + 2 quad + e
    uint32_t qr[C::Q_REGS && !C::F32 ? D / 32 : 1][4];
    uint32_t qrh[C::Q_REGS && C::F32 ? D / 16 : 1][4], qrl[C::Q_REGS && C::F32 ? D / 16 : 1][4];
#pragma unroll 1
    for (int j = -NS; j < 2 * n; ++j) {
      if (j >= 0) {
        cp_wait<NS - 1>();
        __syncwarp();
        if ((j & 1) == 0) {
          // -------- scores of group j / 2
          const int j0 = first + (j >> 1) * GROUP;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt) sc[kt][nt][0] = sc[kt][nt][1] = sc[kt][nt][2] = sc[kt][nt][3] = 0.f;
          if constexpr (!C::F32) {
            if (C::Q_REGS && j == 0) {
#pragma unroll
              for (int kp = 0; kp < D / 32; ++kp) ldsm4(sq + at_rows<RB>(mr, 4 * kp + mat), qr[C::Q_REGS ? kp : 0]);
            }
#pragma unroll
            for (int kp = 0; kp < D / 32; ++kp) {  // two k16 steps
              uint32_t ka[KT][2][4];  // keys 0-7, 8-15 of columns low, then high
#pragma unroll
              for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  ldsm4(use + at_rows<RB>(kt * 16 + (mat & 1) * 8 + mr, 4 * kp + 2 * e + (mat >> 1)), ka[kt][e]);
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt) {
                uint32_t qb[4];
                if constexpr (C::Q_REGS) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) qb[e] = qr[kp][e];
                } else {
                  ldsm4(sq + at_rows<RB>(nt * 8 + mr, 4 * kp + mat), qb);
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                  mma_bf16(sc[kt][nt], ka[kt][0], qb[0], qb[1]);
                  mma_bf16(sc[kt][nt], ka[kt][1], qb[2], qb[3]);
                }
              }
            }
          } else {
            // The tensor core cuts off what it adds to a sum below the sum's last bit: the small
            // products have sums of their own, so that the large one is cut a third as often.
            if (C::Q_REGS && j == 0) {
#pragma unroll
              for (int kp = 0; kp < D / 16; ++kp) {
                uint32_t v[4];
                ldsm4(sq + at_rows<RB>(mr, 4 * kp + mat), v);
#pragma unroll
                for (int z = 0; z < 4; ++z) split(v[z], qrh[C::Q_REGS ? kp : 0][z], qrl[C::Q_REGS ? kp : 0][z]);
              }
            }
            float lh[KT][NTR][4], hl[KT][NTR][4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) lh[kt][nt][e] = hl[kt][nt][e] = 0.f;
#pragma unroll
            for (int kp = 0; kp < D / 16; ++kp) {  // two k8 steps: four chunks of four columns
              uint32_t kh[KT][2][4], kl[KT][2][4];
#pragma unroll
              for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint32_t v[4];
                  ldsm4(use + at_rows<RB>(kt * 16 + (mat & 1) * 8 + mr, 4 * kp + 2 * e + (mat >> 1)), v);
#pragma unroll
                  for (int z = 0; z < 4; ++z) split(v[z], kh[kt][e][z], kl[kt][e][z]);
                }
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt) {
                uint32_t v[4], qh[4], ql[4];
                if constexpr (C::Q_REGS) {
#pragma unroll
                  for (int z = 0; z < 4; ++z) { qh[z] = qrh[kp][z]; ql[z] = qrl[kp][z]; }
                } else {
                  ldsm4(sq + at_rows<RB>(nt * 8 + mr, 4 * kp + mat), v);
#pragma unroll
                  for (int z = 0; z < 4; ++z) split(v[z], qh[z], ql[z]);
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    mma_tf32(hl[kt][nt], kh[kt][e], ql[2 * e], ql[2 * e + 1]);
                    mma_tf32(lh[kt][nt], kl[kt][e], qh[2 * e], qh[2 * e + 1]);
                    mma_tf32(sc[kt][nt], kh[kt][e], qh[2 * e], qh[2 * e + 1]);
                  }
              }
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[kt][nt][e] += lh[kt][nt][e] + hl[kt][nt][e];
          }
          if (j0 < in_lo || j0 + GROUP - 1 > in_hi) {
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // row 8 nt + 2 quad + e sees keys [lo, hi]
                const int p = s.len - s.n + g.rep.of(x.rho0 + min(nt * 8 + quad * 2 + e, x.rows - 1));
                const int hi = g.causal ? min(p, s.len - 1) : s.len - 1;
                const int lo = g.window > 0 ? p - g.window + 1 : 0;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    const int key = j0 + kt * 16 + z * 8 + oct;
                    if (key < lo || key > hi) sc[kt][nt][2 * z + e] = -INFINITY;
                  }
              }
          }
          // -------- probabilities; m where it has to move
          float mx[NTR][2];
          bool grow = false;
#pragma unroll
          for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
              for (int kt = 1; kt < KT; ++kt) v = ptx::max3(v, sc[kt][nt][e], sc[kt][nt][e + 2]);
              mx[nt][e] = v * a.sl2;
              grow |= mx[nt][e] > m[nt][e] + RESCALE_THRESHOLD;
            }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                const float mn = fmaxf(m[nt][e], v);
                const float f = ptx::ex2(m[nt][e] - mn);
                m[nt][e] = mn;
                l[nt][e] *= f;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                  o[d][nt][e] *= f;
                  o[d][nt][e + 2] *= f;
                }
              }
          }
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float p = ptx::ex2(fmaf(sc[kt][nt][e], a.sl2, -m[nt][e & 1]));
                sc[kt][nt][e] = p;
                l[nt][e & 1] += p;
              }
        } else if constexpr (!C::F32) {
          // -------- O^T += V^T P^T
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            uint32_t ph[NTR][2], pl[NTR][2];  // keys low, high
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p0 = sc[kt][nt][2 * e], p1 = sc[kt][nt][2 * e + 1];
                const uint32_t hi = bf2(p0, p1);
                ph[nt][e] = transpose8(hi);
                pl[nt][e] = transpose8(bf2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
              }
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t va[4];  // columns 0-7, 8-15 of keys low, then high
              ldsm4t(use + at_rows<RB>(kt * 16 + (mat >> 1) * 8 + mr, 2 * d + (mat & 1)), va);
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt) {
                mma_bf16(o[d][nt], va, pl[nt][0], pl[nt][1]);
                mma_bf16(o[d][nt], va, ph[nt][0], ph[nt][1]);
              }
            }
          }
        } else {
          uint32_t ph[NTR][2 * KT][2], pl[NTR][2 * KT][2];  // k8 steps: keys quad, quad + 4
#pragma unroll
          for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
            for (int k8 = 0; k8 < 2 * KT; ++k8)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // key quad + 4 e, row oct: in lane 4 key + row / 2, value row & 1
                const int from = (quad + 4 * e) * 4 + (oct >> 1);
                const float p0 = __shfl_sync(0xffffffffu, sc[k8 >> 1][nt][2 * (k8 & 1)], from);
                const float p1 = __shfl_sync(0xffffffffu, sc[k8 >> 1][nt][2 * (k8 & 1) + 1], from);
                split(__float_as_uint(oct & 1 ? p1 : p0), ph[nt][k8][e], pl[nt][k8][e]);
              }
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t vh[2 * KT][4], vl[2 * KT][4];  // columns oct, oct + 8 of key quad, then of key quad + 4
#pragma unroll
            for (int k8 = 0; k8 < 2 * KT; ++k8)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int col = d * 16 + (e & 1) * 8 + oct, key = k8 * 8 + (e >> 1) * 4 + quad;
                split(lds32(use + at_v32<RB>(key, col >> 2) + (col & 3) * 4), vh[k8][e], vl[k8][e]);
              }
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt) {
              // a sum per group, added to O in fp32: O itself is not cut at every step
              float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int k8 = 0; k8 < 2 * KT; ++k8) {
                mma_tf32(add, vl[k8], ph[nt][k8][0], ph[nt][k8][1]);
                mma_tf32(add, vh[k8], pl[nt][k8][0], pl[nt][k8][1]);
              }
#pragma unroll
              for (int k8 = 0; k8 < 2 * KT; ++k8) mma_tf32(add, vh[k8], ph[nt][k8][0], ph[nt][k8][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[d][nt][e] += add[e];
            }
          }
        }
        __syncwarp();  // the slot is read
        use = use + C::SLOT == ring + NS * C::SLOT ? ring : use + C::SLOT;
      }
      load(j + NS);
    }
    cp_wait<0>();
    __syncwarp();  // (every lane's copies have landed: the ring may be used for what comes next)

    // ---- this warp's sums into its shared memory
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int r = nt * 8 + quad * 2 + e;
        if (oct == 0) ml_sh[warp][r] = make_float2(m[nt][e], v);
        float* const to = reinterpret_cast<float*>(mine) + r * C::OS + oct;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          to[d * 16] = o[d][nt][e];
          to[d * 16 + 8] = o[d][nt][e + 2];
        }
      }
    fin = {s.row0, x.rho0, x.rows, seg.head, walk.p.ender,
           (seg.starts ? PART_STARTS : 0) | (seg.ends ? PART_ENDS : 0), 2 * worker + seg.slot};
    __syncwarp();
    held = seg.slot == 0 && walk.done() && !(seg.starts && seg.ends);
    if (!held) {
      finish<C, D>(a, fin, smem, ml_sh, warp, warp, lane, 32);
      __syncwarp();
    }
  }

  // ---- all warps with parts of one and the same item: one result (or part) for the CTA
  if (lane == 0 && walk.moved) {
    item_sh[warp].w = held;
    ends_sh[warp] = fin.flags;
  }
  __syncthreads();
  bool same = item_sh[0].w == 1;
  int last = 0;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) {
    const int4 p = item_sh[0], q = item_sh[w];
    if (q.w == 2) continue;  // no part
    same = same && last == w - 1 && q.w == 1 && q.x == p.x && q.y == p.y && q.z == p.z;
    last = w;
  }
  if (!held) return;
  same = same && last > 0;
  if (same) {
    fin.flags = (ends_sh[0] & PART_STARTS) | (ends_sh[last] & PART_ENDS) | PART_JOINED;
    fin.slot = 2 * blockIdx.x * WARPS;
    // (the join counts the workers up to the one that ends an item: nothing of the others)
    if (warp > 0 && lane < R && (fin.flags & PART_ENDS))
      a.part.ml[(size_t)2 * worker * R + lane] = make_float2(-FLT_MAX, 0.f);
  }
  finish<C, D>(a, fin, smem, ml_sh, same ? 0 : warp, same ? last : warp, same ? tid : lane, same ? 32 * (last + 1) : 32);
}

// An item that several workers did parts of: the worker in whose part it starts left the
// first one (at most one such per worker, its last item: slot 1, or 0 if it is its first
// too), those after it the others in their slots 0, up to the one that ends it; a CTA all
// inside the item left one part for its workers, in the first one's slot. Blocks (c, y) stand
// for CTA c. At most one of its open items goes on beyond it: the blocks share out its rows,
// and their warps its parts. An item that ends in the CTA has few parts: a warp of each block
// joins them. Lanes are columns. Sums are merged in a fixed order. Most blocks find nothing
// open and go. (One sequence of 16384 tokens, 114 parts of 4 rows: 11 us; nothing open: 3.5.)
constexpr int JOIN_WARPS = 4;
constexpr int JOIN_THREADS = 32 * JOIN_WARPS;

// columns 4 col .. of row r of the item: written from its sums
__device__ __forceinline__ void join_row(const JoinArgs& a, const Left& f, int r, int col, const Sum& x) {
  const int rho = f.rho0 + r, token = a.rep.of(rho);
  x.write(a.O, a.LSE, (size_t)(f.row0 + token) * a.H + f.head * a.rep.d + rho - token * a.rep.d, col * 4, a.Dv, a.out_bf16);
}

// `where`: the worker of the CTA that left the item open, + 16 if in its slot 1. ALL: by all
// blocks and warps of the CTA, else by the calling warp.
template <bool ALL>
__device__ __forceinline__ void join_item(const JoinArgs& a, int where, int last_worker, int warp, int lane) {
  __shared__ float2 ml[JOIN_THREADS];
  __shared__ float4 acc_sh[JOIN_THREADS];
  const int k = blockIdx.x * a.per + (where & 15), which = where >> 4;
  const Left f = a.part.left[2 * k + which];
  // parts: worker k's, those of the workers after it in its CTA, one of each CTA all inside,
  // those of the last CTA up to the worker that ends the item
  const int end = min(f.ender, last_worker), c0 = blockIdx.x, c1 = end / a.per;
  const int near = (f.flags & PART_JOINED) ? 0 : min(end, c0 * a.per + a.per - 1) - k;
  const int inside = max(0, c1 - c0 - 1);
  const int parts = 1 + near + inside + (c1 > c0 ? end - c1 * a.per + 1 : 0);
  auto slot_of = [&](int p) {
    if (p == 0) return 2 * k + which;
    if (p <= near) return 2 * (k + p);
    p -= near;
    return p <= inside ? 2 * (c0 + p) * a.per : 2 * (c1 * a.per + p - inside - 1);
  };
  const int cols = a.D / 4, side = 32 / cols;  // lanes of a row; rows of a warp
  const int col = lane % cols, sub = lane / cols;
  const int p0 = ALL ? parts * warp / JOIN_WARPS : 0;
  const int p1 = ALL ? parts * (warp + 1) / JOIN_WARPS : parts;
  for (int g = blockIdx.y; g * side < f.rows; g += gridDim.y) {
    const int r = g * side + sub;
    Sum x = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (r < f.rows) {
      constexpr int U = 8;
      for (int p = p0; p < p1; p += U) {
        float2 y[U];
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (p + u < p1) {
            const size_t row = (size_t)slot_of(p + u) * a.R + r;
            y[u] = a.part.ml[row];
            v[u] = *reinterpret_cast<const float4*>(a.part.O + row * a.D + col * 4);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (p + u < p1 && !(y[u].y == 0.f)) x.add(y[u].x, y[u].y, v[u]);
      }
    }
    if (ALL) {
      ml[threadIdx.x] = make_float2(x.M, x.L);
      acc_sh[threadIdx.x] = x.acc;
      __syncthreads();
      for (int w = 1; warp == 0 && w < JOIN_WARPS; ++w)
        x.add(ml[w * 32 + lane].x, ml[w * 32 + lane].y, acc_sh[w * 32 + lane]);
      __syncthreads();
    }
    if (r < f.rows && (!ALL || warp == 0)) join_row(a, f, r, col, x);
  }
}

__global__ void __launch_bounds__(JOIN_THREADS, 5) attend_join_kernel(const __grid_constant__ JoinArgs a) {
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // worker w's open item, if any, in lanes w and w + 16 (slot 0 or 1)
  const int last_worker = a.ctas * a.per - 1;
  int open = 0, ender = 0;
  {
    const int w = lane & 15, slot = 2 * (blockIdx.x * a.per + w) + (lane >> 4);
    if (w < a.per) {
      const Left& f = a.part.left[slot];
      open = (f.flags & (PART_STARTS | PART_ENDS)) == PART_STARTS;
      ender = f.ender;
    }
  }
  const int first_after = (blockIdx.x + 1) * a.per;
  const unsigned far = __ballot_sync(0xffffffffu, open && ender >= first_after);
  const unsigned near_by = __ballot_sync(0xffffffffu, open && ender < first_after);
  if (far) join_item<true>(a, __ffs(far) - 1, last_worker, warp, lane);
  const unsigned me = near_by & (0x10001u << warp);
  if (warp < a.per && me) join_item<false>(a, __ffs(me) - 1, last_worker, warp, lane);
}

// The same where a CTA is a worker and items are tall: at most an open item per CTA, few of
// them with many parts or many with few. Every block lists the open items (they are few
// enough to look at all of them), and the rows of all items together are shared out evenly
// among the warps of the grid, a run of rows each: four rows at a time with two parts of
// each on the way, or, where there are no more rows than warps, one row with eight parts.
// (2048 tokens over 16384: 39 MB of parts in 15 us.)
constexpr int TALL_WARPS = 8;
constexpr int TALL_BLOCKS = 2;  // per SM
template <int ROWS, int U>
__device__ __forceinline__ void join_rows(const JoinArgs& a, const Left* open, const int* first, int n, int lane) {
  const int cols = a.D / 4, side = 32 / cols;
  const int col = lane % cols, sub = lane / cols;
  const int warps = gridDim.x * TALL_WARPS, run = (first[n] + warps - 1) / warps;
  int at = (blockIdx.x * TALL_WARPS + (threadIdx.x >> 5)) * run;
  const int end = min(first[n], at + run);
  while (at < end) {
    int lo = 0, hi = n;  // the item of row `at`
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= at) lo = mid; else hi = mid;
    }
    const Left f = open[lo];
    const int c0 = f.pad[0], parts = f.ender - c0 + 1;
    const int r_end = min(end, first[lo + 1]) - first[lo];
    for (int r = at - first[lo]; r < r_end; r += ROWS * side) {
      Sum x[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) x[i] = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int p = 0; p < parts; p += U) {
        float2 y[U][ROWS];
        float4 v[U][ROWS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // (past the last part: that part again, not counted)
          const size_t slot = p + u == 0 ? f.pad[1] : 2 * (c0 + min(p + u, parts - 1));
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const size_t row = slot * a.R + min(r + i * side + sub, r_end - 1);
            y[u][i] = a.part.ml[row];
            v[u][i] = *reinterpret_cast<const float4*>(a.part.O + row * a.D + col * 4);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            if (p + u < parts && !(y[u][i].y == 0.f)) x[i].add(y[u][i].x, y[u][i].y, v[u][i]);
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (r + i * side + sub < r_end) join_row(a, f, r + i * side + sub, col, x[i]);
    }
    at = first[lo] + r_end;
  }
}

__global__ void __launch_bounds__(32 * TALL_WARPS, TALL_BLOCKS) attend_join_tall_kernel(const __grid_constant__ JoinArgs a) {
  ptx::grid_dependency_wait();
  __shared__ Left open[TALL_CTAS];
  __shared__ int first[TALL_CTAS + 1];
  __shared__ int2 sums[TALL_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = 0, rows = 0;  // open items and their rows so far
  for (int c0 = 0; c0 < a.ctas; c0 += 32 * TALL_WARPS) {
    const int c = c0 + tid;
    Left f = {};
    if (c < a.ctas) {
      const Left f0 = a.part.left[2 * c], f1 = a.part.left[2 * c + 1];
      constexpr int OPEN = PART_STARTS | PART_ENDS;
      const bool second = (f1.flags & OPEN) == PART_STARTS;
      f = second ? f1 : f0;
      if ((f.flags & OPEN) != PART_STARTS) f.rows = 0;
      f.pad[0] = c;
      f.pad[1] = 2 * c + second;
    }
    const int is = f.rows > 0;
    int k = is, r = f.rows;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, k, d), v = __shfl_up_sync(0xffffffffu, r, d);
      if (lane >= d) { k += u; r += v; }
    }
    if (lane == 31) sums[warp] = make_int2(k, r);
    __syncthreads();
    int2 before = make_int2(n, rows);
    for (int w = 0; w < TALL_WARPS; ++w) {
      if (w < warp) { before.x += sums[w].x; before.y += sums[w].y; }
      n += sums[w].x;
      rows += sums[w].y;
    }
    if (is) {
      open[before.x + k - is] = f;
      first[before.x + k - is] = before.y + r - f.rows;
    }
    __syncthreads();
  }
  if (tid == 0) first[n] = rows;
  __syncthreads();
  if (n == 0) return;
  if (rows > 2 * (int)gridDim.x * TALL_WARPS) join_rows<4, 2>(a, open, first, n, lane);
  else join_rows<1, 8>(a, open, first, n, lane);
}

template <typename E, int D, int NTR>
fa_status run(RowsArgs& a, cudaStream_t s) {
  using C = RowsCfg<E, D, NTR>;
  auto* kernel = attend_rows_kernel<E, D, NTR>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return failed();
  const int ctas = host::sm_count() * C::CTAS_PER_SM;
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas * WARPS, C::R, D), s) != cudaSuccess) return failed();
  a.part = partials_at(w, ctas * WARPS, C::R, D);
  a.g.R = C::R;
  a.g.u_shift = log2_of(C::GROUP);
  a.g.start = 4;  // groups: looking up an item's first pages and rows takes about as long
  a.g.snap = 4;
  fa_status st;
  {
    host::KernelTimer t("attend_rows", s);
    st = launch(kernel, ctas, NTHREADS, C::SMEM, s, a);
  }
  if (st == FA_OK) {
    const JoinArgs j = {a.part, a.O, a.LSE, ctas, WARPS, C::R, D, a.H, a.c.D, a.out_bf16, a.g.rep};
    st = launch_join(j, s);
  }
  if (host::scratch_free(w, s) != cudaSuccess) st = failed();
  return st;
}

}  // namespace

fa_status launch_join(const JoinArgs& a, cudaStream_t s) {
  host::KernelTimer t("attend_join", s);
  return launch_dependent(attend_join_kernel, dim3(a.ctas, a.R / 2), JOIN_THREADS, s, a);
}

fa_status launch_join_tall(const JoinArgs& a, cudaStream_t s) {
  host::KernelTimer t("attend_join", s);
  return launch_dependent(attend_join_tall_kernel, TALL_BLOCKS * host::sm_count(), 32 * TALL_WARPS, s, a);
}

fa_status launch_attend_rows(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                             const fakv_cache& c, const fakv_tokens& p, cudaStream_t s) {
  RowsArgs a = {};
  a.c = c;
  a.q = q;
  a.O = O;
  a.LSE = LSE;
  a.cu = cu;
  a.slots = slots;
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.plane = p.plane;
  a.shift = log2_of(c.page_size);
  a.q_token = p.q_token;
  a.q_head = p.q_head;
  const int rep = p.H / c.HKV;
  a.g.rep = div_by(rep);
  a.g.causal = p.causal;
  a.g.window = p.window;
  a.sl2 = p.scale * LOG2E;
  a.out_bf16 = p.out_dtype == FA_BF16;
  // Items of 8, 16 or (fp32: a bf16 cache's rows above 16 are the tensor-core tiles') 32 rows: what
  // a sequence's rows fit on average.
  const long long rows = ((long long)p.T * rep + p.B - 1) / p.B;
  if (c.dtype == FA_BF16) {
    if (c.D <= 64) return rows <= 8 ? run<__nv_bfloat16, 64, 1>(a, s) : run<__nv_bfloat16, 64, 2>(a, s);
    return rows <= 8 ? run<__nv_bfloat16, 128, 1>(a, s) : run<__nv_bfloat16, 128, 2>(a, s);
  }
  if (c.D <= 64) return rows <= 8 ? run<float, 64, 1>(a, s) : rows <= 16 ? run<float, 64, 2>(a, s) : run<float, 64, 4>(a, s);
  return rows <= 8 ? run<float, 128, 1>(a, s) : rows <= 16 ? run<float, 128, 2>(a, s) : run<float, 128, 4>(a, s);
}

}  // namespace kv
}  // namespace fa
