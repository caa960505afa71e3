// kv_rows.cuh -- what the kernels of few rows share (a warp is a worker, mma.sync): copies,
// fragments, an item's sums and how they are put together in a CTA.
#pragma once
#include <cfloat>
#include <cmath>
#include "kv_sched.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int WARPS = 4;
constexpr int NTHREADS = 32 * WARPS;

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
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
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
template <typename C, int D, typename A>
__device__ __forceinline__ void finish(const A& a, const Finish& f, const uint8_t* smem,
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

// What a CTA's warps are about when their parts are done (in shared memory).
template <int R>
struct Ends {
  float2 ml[WARPS][R];
  int4 item[WARPS];  // b, tile, head, and 1: held, 2: no part, 0: neither
  int ends[WARPS];   // a held item's PART_STARTS, PART_ENDS
};

// A worker's only item, not done whole, is held until the others are done: where all warps of
// the CTA have parts of one and the same item, they leave one result (or part) for the CTA.
template <typename C, int D, typename A>
__device__ __forceinline__ void finish_held(const A& a, Finish fin, bool held, bool moved, const uint8_t* smem,
                                            Ends<C::R>& sh) {
  constexpr int R = C::R;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x * WARPS + warp;
  if (lane == 0 && moved) {
    sh.item[warp].w = held;
    sh.ends[warp] = fin.flags;
  }
  __syncthreads();
  bool same = sh.item[0].w == 1;
  int last = 0;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) {
    const int4 p = sh.item[0], q = sh.item[w];
    if (q.w == 2) continue;  // no part
    same = same && last == w - 1 && q.w == 1 && q.x == p.x && q.y == p.y && q.z == p.z;
    last = w;
  }
  if (!held) return;
  same = same && last > 0;
  if (same) {
    fin.flags = (sh.ends[0] & PART_STARTS) | (sh.ends[last] & PART_ENDS) | PART_JOINED;
    fin.slot = 2 * blockIdx.x * WARPS;
    // (the join counts the workers up to the one that ends an item: nothing of the others)
    if (warp > 0 && lane < R && (fin.flags & PART_ENDS))
      a.part.ml[(size_t)2 * worker * R + lane] = make_float2(-FLT_MAX, 0.f);
  }
  finish<C, D>(a, fin, smem, sh.ml, same ? 0 : warp, same ? last : warp, same ? tid : lane, same ? 32 * (last + 1) : 32);
}

}  // namespace
}  // namespace kv
}  // namespace fa
