// kv_rows.cu -- attention over the paged cache for few rows per sequence (decoding), and
// for fp32 caches: K and V streamed once, mma.sync.
//
// Few rows read many keys: 4 D flops per row against 4 D bytes (bf16) per key, so up to a
// few dozen rows the work is bound by HBM. A CTA (4 warps) walks its part of the work line
// (kv_sched.cuh) in units of 64 keys, 16 per warp: a warp has its own ring of 16-key
// stages, filled with cp.async (any page size and stride, no copy descriptor to build on
// the host), its own running maximum, sum and O, and meets the others only at the end of an
// item: the loop has no CTA barrier. A 16-row tile of mma.sync holds the rows (two
// for up to 32): even with 4 rows in it, the tensor work per 16 keys is a third of the time
// their bytes take, whereas tcgen05's 128-row tile would mean a TMEM round trip per tile
// for the same bytes.
//
//   scores  S = Q K^T: bf16 m16n8k16, fp32 sums. fp32 caches: x = hi + lo with tf32 terms,
//           hi hi + hi lo + lo hi (m16n8k8).
//   softmax online in the exp2 domain; m moves only when it would grow by more than 8
//           (the sums stay exact: every exponential of an item is taken against the same m
//           as its O).
//   O += P V  bf16: P = hi + lo, two bf16 terms, so that P's rounding (2^-9) does not add
//           to the output's: the second product is free under the memory time.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include "kv_sched.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int WARPS = 4;
constexpr int NTHREADS = 32 * WARPS;
constexpr int GROUP = 16;             // keys per warp step
constexpr int UNIT = GROUP * WARPS;   // keys per unit

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

template <typename E, int D, int MT>
struct RowsCfg {
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int R = 16 * MT;
  static constexpr int RB = D * (int)sizeof(E);   // bytes of a K / V / Q row
  static constexpr int CH = RB / 16;              // 16-byte chunks of it
  static constexpr int STAGE = 2 * GROUP * RB;    // K and V of a group
  static constexpr int WARP_BYTES = 24576 * (F32 && D == 128 ? 2 : 1);
  static constexpr int S = WARP_BYTES / STAGE;    // stages of a warp's ring
  static constexpr int OS = D + 8;                // floats of a merged O row (bank spread)
  static constexpr int Q_BYTES = R * RB;
  static constexpr int SMEM = WARPS * WARP_BYTES + Q_BYTES;
  static constexpr int CTAS_PER_SM = SMEM > 110 * 1024 ? 1 : 2;
  static_assert(S >= 3 && R * OS * 4 <= WARP_BYTES, "a warp's ring also holds its O for the merge");
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
// x = hi + lo: hi the value rounded to tf32's 11 significant bits, lo the rest, rounded too
// (the tensor core drops the 13 low bits, so half of their step is added first; truncated
// terms would all err to one side: O was 2.7e-6 off instead of a third of that)
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
  hi = (x + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) + 0x1000u;
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
  return (uint32_t)(row * RB + ((chunk ^ (((row >> 1) & 3) << 1)) << 4));
}

template <typename E, int D, int MT>
__global__ void __launch_bounds__(NTHREADS, RowsCfg<E, D, MT>::CTAS_PER_SM)
    attend_rows_kernel(const __grid_constant__ RowsArgs a) {
  using C = RowsCfg<E, D, MT>;
  constexpr int RB = C::RB, CH = C::CH, R = C::R, S = C::S;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ PlanShared plan;
  __shared__ float2 ml_sh[WARPS][R];
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, qrow = lane >> 2;
  const fakv_cache& c = a.c;
  const Geo& g = a.g;
  const Part part = find_part<NTHREADS>(g, c, a.cu, a.slots, a.B, a.T, reinterpret_cast<int*>(smem), plan,
                                        blockIdx.x, gridDim.x);
  if (tid < 2) {
    a.part.left[2 * blockIdx.x + tid].flags = 0;  // (an entry of this CTA's is written below)
  }
  if (part.units == 0) return;
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::WARP_BYTES;
  const uint32_t sq = ptx::smem_u32(smem) + WARPS * C::WARP_BYTES;
  const int dv_chunks = c.D * (int)sizeof(E) / 16;
  const E* const Kp = static_cast<const E*>(c.K) + a.plane * c.plane_stride;
  const E* const Vp = static_cast<const E*>(c.V) + a.plane * c.plane_stride;

  Walk walk(part);
  Seg seg;
  while (walk.next(g, c, a.cu, a.slots, a.T, seg)) {
    const Seq& s = seg.s;
    const Tile& x = seg.x;
    const int head = seg.head;

    // ---- q rows into shared memory (zeros behind the item's rows and the tensor's columns)
    for (int i = tid; i < R * CH; i += NTHREADS) {
      const int r = i / CH, ch = i % CH;
      const int rho = x.rho0 + r;
      const bool in = r < x.rows && ch < dv_chunks;
      const E* src = static_cast<const E*>(a.q);
      if (in)
        src += (s.row0 + rho / g.rep) * a.q_token + (head * g.rep + rho % g.rep) * a.q_head + ch * (16 / (int)sizeof(E));
      cp16(sq + at_rows<RB>(r, ch), src, in);
    }
    cp_commit();

    // ---- this warp's groups of keys: g0, g0 + WARPS, ...
    const int g_end = min((seg.k0 + seg.n) * WARPS, (x.hi + GROUP - 1) / GROUP);
    const int g0 = max(seg.k0 * WARPS, x.lo / GROUP);
    const int gw = g0 + ((warp - g0) & (WARPS - 1));
    const int n = gw < g_end ? (g_end - gw + WARPS - 1) / WARPS : 0;
    // Pages of the next 32 groups, a group per lane (two pages where they hold 8 tokens),
    // and of the 32 after those: look-ups are never waited for in the loop.
    const int* const row = c.table + (long long)s.slot * c.table_stride;
    auto lookup = [&](int i, int& p0, int& p1) {
      p0 = p1 = -1;
      if (i < n) {
        const int j = (gw + i * WARPS) * GROUP;
        if (a.shift > 3) {
          p0 = p1 = row[j >> a.shift];
        } else {  // (a half that no row sees is not looked up)
          p0 = j + 8 > x.lo ? row[j >> 3] : 0;
          p1 = j + 8 < x.hi ? row[(j + 8) >> 3] : 0;
        }
        if ((unsigned)p0 >= (unsigned)c.num_pages || (unsigned)p1 >= (unsigned)c.num_pages)
          raise(c.status, FAKV_BAD_PAGE);
      }
    };
    int pg0, pg1, nx0, nx1;
    lookup(lane, pg0, pg1);
    lookup(32 + lane, nx0, nx1);
    auto load = [&](int i) {
      if (i < n) {
        if (i > 0 && (i & 31) == 0) {
          pg0 = nx0;
          pg1 = nx1;
          lookup(i + 32 + lane, nx0, nx1);
        }
        const int p[2] = {__shfl_sync(0xffffffffu, pg0, i & 31), __shfl_sync(0xffffffffu, pg1, i & 31)};
        const int j0 = (gw + i * WARPS) * GROUP;
        const uint32_t st = ring + (i % S) * C::STAGE;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool page_ok = (unsigned)p[h] < (unsigned)c.num_pages;
          const long long base = page_ok ? p[h] * c.page_stride + ((j0 + 8 * h) & (c.page_size - 1)) * c.token_stride +
                                               head * c.head_stride
                                         : 0;
#pragma unroll
          for (int k = 0; k < 8 * CH / 32; ++k) {
            const int r = (k * 32 + lane) / CH, ch = (k * 32 + lane) % CH;
            const int j = j0 + 8 * h + r;
            // nothing that no row sees is read: it may hold anything
            const bool in = page_ok && j >= x.lo && j < x.hi && ch < dv_chunks;
            const long long off = in ? base + r * c.token_stride + ch * (16 / (int)sizeof(E)) : 0;
            cp16(st + at_rows<RB>(8 * h + r, ch), Kp + off, in);
            if constexpr (C::F32) cp16(st + GROUP * RB + at_v32<RB>(8 * h + r, ch), Vp + off, in);
            else cp16(st + GROUP * RB + at_rows<RB>(8 * h + r, ch), Vp + off, in);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(i);

    // ---- rows' bounds: row qrow + 8 h + 16 mt sees keys [lo_r, hi_r]
    int lo_r[MT][2], hi_r[MT][2];
    float m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = min(mt * 16 + h * 8 + qrow, x.rows - 1);
        const int p = s.len - s.n + (x.rho0 + r) / g.rep;
        hi_r[mt][h] = g.causal ? min(p, s.len - 1) : s.len - 1;
        lo_r[mt][h] = g.window > 0 ? p - g.window + 1 : 0;
        m[mt][h] = -FLT_MAX;
        l[mt][h] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < D / 8; ++d) o[mt][d][0] = o[mt][d][1] = o[mt][d][2] = o[mt][d][3] = 0.f;
    }
    // keys that every row sees need no mask
    int in_lo, in_hi;
    {
      const int pa = s.len - s.n + x.rho0 / g.rep, pb = s.len - s.n + (x.rho0 + x.rows - 1) / g.rep;
      in_hi = g.causal ? min(pa, s.len - 1) : s.len - 1;
      in_lo = g.window > 0 ? pb - g.window + 1 : 0;
    }
    cp_wait<S - 1>();  // q (committed before the first group)
    __syncthreads();

    for (int i = 0; i < n; ++i) {
      cp_wait<S - 2>();
      __syncwarp();  // the group is here, and every lane has read the one before it:
      load(i + S - 1);  // its stage is filled again
      const uint32_t sk = ring + (i % S) * C::STAGE, sv = sk + GROUP * RB;
      const int j0 = (gw + i * WARPS) * GROUP;
      float sc[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
      const int mat = lane >> 3, mr = lane & 7;
      if constexpr (!C::F32) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kb[4];  // keys 0-7: k low, high; keys 8-15: k low, high
          ldsm4(sk + at_rows<RB>((mat >> 1) * 8 + mr, 2 * ks + (mat & 1)), kb);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t qa[4];
            ldsm4(sq + at_rows<RB>(mt * 16 + (mat & 1) * 8 + mr, 2 * ks + (mat >> 1)), qa);
            mma_bf16(sc[mt][0], qa, kb[0], kb[1]);
            mma_bf16(sc[mt][1], qa, kb[2], kb[3]);
          }
        }
      } else {
        // The tensor core cuts off what it adds to a sum below the sum's last bit: the small
        // products have sums of their own, so that the large one is cut a third as often.
        float small[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) small[mt][nt][0] = small[mt][nt][1] = small[mt][nt][2] = small[mt][nt][3] = 0.f;
#pragma unroll
        for (int kp = 0; kp < D / 16; ++kp) {  // two k8 steps: four chunks of four
          uint32_t kh[2][4], kl[2][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            uint32_t v[4];
            ldsm4(sk + at_rows<RB>(nt * 8 + mr, 4 * kp + mat), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) split(v[e], kh[nt][e], kl[nt][e]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t v[4], qh[4], ql[4];
              ldsm4(sq + at_rows<RB>(mt * 16 + (mat & 1) * 8 + mr, 4 * kp + 2 * e + (mat >> 1)), v);
#pragma unroll
              for (int z = 0; z < 4; ++z) split(v[z], qh[z], ql[z]);
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                mma_tf32(small[mt][nt], qh, kl[nt][2 * e], kl[nt][2 * e + 1]);
                mma_tf32(small[mt][nt], ql, kh[nt][2 * e], kh[nt][2 * e + 1]);
                mma_tf32(sc[mt][nt], qh, kh[nt][2 * e], kh[nt][2 * e + 1]);
              }
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] += small[mt][nt][e];
      }
      if (j0 < in_lo || j0 + GROUP - 1 > in_hi) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + nt * 8 + quad * 2 + (e & 1);
              if (j < lo_r[mt][e >> 1] || j > hi_r[mt][e >> 1]) sc[mt][nt][e] = -INFINITY;
            }
      }
      // maxima of the rows, and m where it has to move
      bool grow = false;
      float mx[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = fmaxf(fmaxf(sc[mt][0][2 * h], sc[mt][0][2 * h + 1]), fmaxf(sc[mt][1][2 * h], sc[mt][1][2 * h + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          mx[mt][h] = v * a.sl2;
          grow |= mx[mt][h] > m[mt][h] + RESCALE_THRESHOLD;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[mt][h], mx[mt][h]);
            const float f = ptx::ex2(m[mt][h] - mn);
            m[mt][h] = mn;
            l[mt][h] *= f;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              o[mt][d][2 * h] *= f;
              o[mt][d][2 * h + 1] *= f;
            }
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = ptx::ex2(fmaf(sc[mt][nt][e], a.sl2, -m[mt][e >> 1]));
            sc[mt][nt][e] = p;
            l[mt][e >> 1] += p;
          }
      if constexpr (!C::F32) {
        uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // rows r, r + 8 of keys 0-7, then of keys 8-15
            const float p0 = sc[mt][k >> 1][2 * (k & 1)], p1 = sc[mt][k >> 1][2 * (k & 1) + 1];
            ph[mt][k] = bf2(p0, p1);
            pl[mt][k] = bf2(p0 - __uint_as_float(ph[mt][k] << 16), p1 - __uint_as_float(ph[mt][k] & 0xffff0000u));
          }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t vb[4];  // columns 0-7: keys low, high; columns 8-15: keys low, high
          ldsm4t(sv + at_rows<RB>((mat & 1) * 8 + mr, 2 * d + (mat >> 1)), vb);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(o[mt][2 * d], pl[mt], vb[0], vb[1]);
            mma_bf16(o[mt][2 * d + 1], pl[mt], vb[2], vb[3]);
            mma_bf16(o[mt][2 * d], ph[mt], vb[0], vb[1]);
            mma_bf16(o[mt][2 * d + 1], ph[mt], vb[2], vb[3]);
          }
        }
      } else {
        // the eight keys of a k step in the order that a thread's scores have them: k slots
        // quad and quad + 4 are keys 2 quad and 2 quad + 1
        uint32_t ph[MT][2][4], pl[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              split(__float_as_uint(sc[mt][nt][(k & 1) * 2 + (k >> 1)]), ph[mt][nt][k], pl[mt][nt][k]);
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          const int col = d * 8 + qrow;
          uint32_t vh[2][2], vl[2][2];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              split(lds32(sv + at_v32<RB>(nt * 8 + 2 * quad + e, col >> 2) + (col & 3) * 4), vh[nt][e], vl[nt][e]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // a sum per group, added to O in fp32: O itself is not cut at every step
            float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              mma_tf32(add, pl[mt][nt], vh[nt][0], vh[nt][1]);
              mma_tf32(add, ph[mt][nt], vl[nt][0], vl[nt][1]);
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma_tf32(add, ph[mt][nt], vh[nt][0], vh[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][d][e] += add[e];
          }
        }
      }
    }
    cp_wait<0>();
    __syncthreads();

    // ---- the warps' results through shared memory (each in its own ring)
    {
      float* mine = reinterpret_cast<float*>(smem + warp * C::WARP_BYTES);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = l[mt][h];
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          const int r = mt * 16 + h * 8 + qrow;
          if (quad == 0) ml_sh[warp][r] = make_float2(m[mt][h], v);
#pragma unroll
          for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2*>(mine + r * C::OS + d * 8 + quad * 2) =
                make_float2(o[mt][d][2 * h], o[mt][d][2 * h + 1]);
        }
    }
    __syncthreads();
    const bool whole = seg.starts && seg.ends;
    const int slot = 2 * blockIdx.x + seg.slot;
    for (int k = tid; k < x.rows * (D / 4); k += NTHREADS) {
      const int r = k / (D / 4), col = k % (D / 4) * 4;
      float M = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml_sh[w][r].x);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ptx::ex2(ml_sh[w][r].x - M);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem + w * C::WARP_BYTES) + r * C::OS + col);
        L += f * ml_sh[w][r].y;
        acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
      }
      if (whole) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int rho = x.rho0 + r;
        const size_t at = (size_t)(s.row0 + rho / g.rep) * a.H + head * g.rep + rho % g.rep;
        if (col == 0) a.LSE[at] = L > 0.f ? (M + log2f(L)) * LN2 : -INFINITY;
        if (col < c.D) {
          if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + at * c.D + col) =
                make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(a.O) + at * c.D + col) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
      } else {
        *reinterpret_cast<float4*>(a.part.O + ((size_t)slot * R + r) * D + col) = acc;
        if (col == 0) a.part.ml[(size_t)slot * R + r] = make_float2(M, L);
      }
    }
    if (!whole && tid == 0)
      a.part.left[slot] = {PART_VALID | (seg.starts ? PART_STARTS : 0) | (seg.ends ? PART_ENDS : 0), s.row0, x.rho0, x.rows,
                           head, {0, 0, 0}};
    __syncthreads();  // the rings are read: the next item may fill them
  }
}

// An item that several CTAs did parts of: the CTA in whose part it starts left the first
// one (at most one such per CTA, its last item: slot 1, or 0 if it is its first too), the
// following CTAs the others in their slots 0, up to the one that ends it. Blocks (c, y)
// join the item that CTA c left open, y sharing out its rows. A block's threads stand
// for the columns, for rows, and, where there are many parts, for shares of the parts, which
// are merged in order.
constexpr int JOIN_THREADS = 256;
constexpr int JOIN_BLOCKS = 32;

struct Sum {  // sums of exponentials taken against the maximum M
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
};

__global__ void __launch_bounds__(JOIN_THREADS) attend_join_kernel(const __grid_constant__ JoinArgs a) {
  ptx::grid_dependency_wait();
  __shared__ int parts_sh;
  __shared__ float2 ml[JOIN_THREADS];
  __shared__ float4 acc_sh[JOIN_THREADS];
  const int cta = blockIdx.x, tid = threadIdx.x;
  constexpr int OPEN = PART_STARTS | PART_ENDS;
  const int open0 = a.part.left[2 * cta].flags & OPEN, open1 = a.part.left[2 * cta + 1].flags & OPEN;
  if (open0 != PART_STARTS && open1 != PART_STARTS) return;
  const int which = open1 == PART_STARTS;
  const Left f = a.part.left[2 * cta + which];
  if (tid == 0) parts_sh = a.ctas;
  __syncthreads();
  for (int k = cta + 1 + tid; k < a.ctas; k += JOIN_THREADS)
    if (a.part.left[2 * k].flags & PART_ENDS) { atomicMin(&parts_sh, k); break; }
  __syncthreads();
  const int parts = parts_sh - cta + 1;  // slot 2 cta + which, then 2 (cta + 1), ...
  const int cols = a.D / 4, groups = JOIN_THREADS / cols;
  int shares = 1;
  while (shares < groups && shares * 4 < parts) shares *= 2;
  const int side = groups / shares;  // rows at a time
  const int col = tid % cols, r = tid / cols % side, share = tid / (cols * side);
  const int p0 = parts * share / shares, p1 = parts * (share + 1) / shares;
  for (int r0 = blockIdx.y * side; r0 < f.rows; r0 += gridDim.y * side) {
    Sum x = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    const bool mine = r0 + r < f.rows;
    if (mine) {
      constexpr int U = 4;
      for (int p = p0; p < p1; p += U) {
        float2 y[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (p + k < p1) {
            const size_t row = (size_t)(p + k == 0 ? 2 * cta + which : 2 * (cta + p + k)) * a.R + r0 + r;
            y[k] = a.part.ml[row];
            v[k] = *reinterpret_cast<const float4*>(a.part.O + row * a.D + col * 4);
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (p + k < p1) x.add(y[k].x, y[k].y, v[k]);
      }
    }
    ml[tid] = make_float2(x.M, x.L);
    acc_sh[tid] = x.acc;
    __syncthreads();
    if (share == 0 && mine) {
      for (int k = 1; k < shares; ++k) {
        const int at = tid + k * cols * side;
        x.add(ml[at].x, ml[at].y, acc_sh[at]);
      }
      const float inv = x.L > 0.f ? 1.f / x.L : 0.f;
      const int rho = f.rho0 + r0 + r;
      const size_t at = (size_t)(f.row0 + rho / a.rep) * a.H + f.head * a.rep + rho % a.rep;
      if (col == 0) a.LSE[at] = x.L > 0.f ? (x.M + log2f(x.L)) * LN2 : -INFINITY;
      if (col * 4 < a.Dv) {
        if (a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + at * a.Dv + col * 4) =
              make_uint2(bf2(x.acc.x * inv, x.acc.y * inv), bf2(x.acc.z * inv, x.acc.w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.O) + at * a.Dv + col * 4) =
              make_float4(x.acc.x * inv, x.acc.y * inv, x.acc.z * inv, x.acc.w * inv);
      }
    }
    __syncthreads();
  }
}

template <typename E, int D, int MT>
fa_status run(RowsArgs& a, cudaStream_t s) {
  using C = RowsCfg<E, D, MT>;
  auto* kernel = attend_rows_kernel<E, D, MT>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return FA_ERR_CUDA;
  const int ctas = host::sm_count() * C::CTAS_PER_SM;
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas, C::R, D), s) != cudaSuccess) return FA_ERR_CUDA;
  a.part = partials_at(w, ctas, C::R, D);
  a.g.R = C::R;
  a.g.U = UNIT;
  fa_status st = FA_OK;
  {
    host::KernelTimer t("attend_rows", s);
    kernel<<<ctas, NTHREADS, C::SMEM, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) st = FA_ERR_CUDA;
  }
  if (st == FA_OK) {
    const JoinArgs j = {a.part, a.O, a.LSE, ctas, C::R, D, a.H, a.g.rep, a.c.D, a.out_bf16};
    st = launch_join(j, s);
  }
  if (host::scratch_free(w, s) != cudaSuccess && st == FA_OK) st = FA_ERR_CUDA;
  return st;
}

}  // namespace

fa_status launch_join(const JoinArgs& a, cudaStream_t s) {
  host::KernelTimer t("attend_join", s);
  return launch_programmatic(attend_join_kernel, dim3(a.ctas, std::min((a.R + 3) / 4, JOIN_BLOCKS)), dim3(JOIN_THREADS), s, a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
  a.g.rep = p.H / c.HKV;
  a.g.causal = p.causal;
  a.g.window = p.window;
  a.sl2 = p.scale * LOG2E;
  a.out_bf16 = p.out_dtype == FA_BF16;
  // one 16-row tile where a sequence's rows fit it on average, else two
  const bool one = (long long)p.T * a.g.rep <= 16ll * p.B;
  if (c.dtype == FA_BF16) {
    if (c.D <= 64) return one ? run<__nv_bfloat16, 64, 1>(a, s) : run<__nv_bfloat16, 64, 2>(a, s);
    return one ? run<__nv_bfloat16, 128, 1>(a, s) : run<__nv_bfloat16, 128, 2>(a, s);
  }
  if (c.D <= 64) return one ? run<float, 64, 1>(a, s) : run<float, 64, 2>(a, s);
  return one ? run<float, 128, 1>(a, s) : run<float, 128, 2>(a, s);
}

}  // namespace kv
}  // namespace fa
