// kv_tiles.cu -- attention over a bf16 paged cache for many rows per sequence (chunks of a
// prompt): TMA from the pages, tcgen05, TMEM.
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
// Measured: 2048 tokens over 16384 (32 query heads on 8 of 128) 337 us with the join, 1530
// TFLOP/s, 0.80 of the measured peak; 8192 tokens of a prompt 385 us, 0.75. A unit of 128 keys
// takes a CTA 2720 clocks, of which its MMAs fill 2240: a tile's softmax (1130 clocks: 62 to
// load the scores, 320 for the maximum, 690 for the exponentials) and the hand-offs on both
// sides of it are longer than the other tile's MMAs. Tried, and slower: two threads to a row
// (640 threads leave 96 registers each: it spilled, 633 us), and P handed over in two halves
// (2820 clocks). An item costs 4 us besides its units (epilogue, first scores), which the
// schedule counts as three units; the start of the kernel 8 us.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include "kv_sched.cuh"

namespace fa {
namespace kv {

static __device__ unsigned int g_kv_status = 0;

namespace {
using namespace ptx;

struct TilesArgs {
  fakv_cache c;
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

template <int D_>
struct TilesCfg {
  static constexpr int D = D_;
  static constexpr int NQ = 2;
  static constexpr int NCB = D / 64;                      // 64-column blocks
  static constexpr uint32_t CB_BYTES = 128u * 128u;       // one block of a 128-row tile
  static constexpr uint32_t TILE_BYTES = NCB * CB_BYTES;
  static constexpr int KST = D == 128 ? 2 : 3;
  static constexpr int VST = 3;
  static constexpr uint32_t EPI_BOX = 32u * 128u;         // a warp's staging: 32 rows x 128 bytes
  static constexpr uint32_t V_STAGE = std::max(TILE_BYTES, 4 * NQ * EPI_BOX);
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t K_OFF = Q_OFF + NQ * TILE_BYTES;
  static constexpr uint32_t V_OFF = K_OFF + KST * TILE_BYTES;
  static constexpr uint32_t SMEM = V_OFF + VST * V_STAGE + 1024;
  static constexpr int SOFTMAX_WARPS = 8, MMA_WARP = 8, KQ_WARP = 9, V_WARP = 10, RELAY_WARP = 11;
  static constexpr uint32_t RELAY_BAR = 3;  // named barrier (1 + q: P_q written)
  static constexpr int THREADS = 384;
  static constexpr uint32_t REGS_SOFTMAX = 216, REGS_CONTROL = 64;
  static_assert(2 * 128 * REGS_SOFTMAX + 128 * REGS_CONTROL <= 384 * 168, "register split exceeds the launch allocation");
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

template <class C>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t sq, uint32_t sk) {
  constexpr uint32_t id = make_idesc(128, 128, FMT_BF16, FMT_BF16, false, false);
#pragma unroll
  for (int kk = 0; kk < C::D / 16; ++kk) {
    const uint32_t off = (kk / 4) * C::CB_BYTES + (kk % 4) * 32;
    mma_f16_ss(d_tmem, make_sdesc(sq + off, 16, SW128_ATOM), make_sdesc(sk + off, 16, SW128_ATOM), id, kk > 0);
  }
}
template <class C, int TERMS>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t sv, bool accumulate) {
  constexpr uint32_t id = make_idesc(128, C::D, FMT_BF16, FMT_BF16, false, true);
#pragma unroll
  for (int term = TERMS - 1; term >= 0; --term)
#pragma unroll
    for (int kk = 0; kk < BLOCK_N / 16; ++kk)
      mma_f16_ts(o_tmem, p_tmem + term * 64 + kk * 8, make_sdesc(sv + kk * 16 * 128, C::CB_BYTES, SW128_ATOM), id,
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

template <int D, int TERMS>
__global__ void __launch_bounds__(TilesCfg<D>::THREADS, 1)
    attend_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TilesArgs a) {
  using C = TilesCfg<D>;
  constexpr int NQ = C::NQ, KST = C::KST, VST = C::VST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_q[NQ], bar_qfree[NQ], bar_kfull[KST], bar_kempty[KST], bar_vfull[VST],
      bar_vempty[VST], bar_grant[NQ], bar_s[NQ], bar_o[NQ], bar_join, bar_drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, stuck_sh;
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
      mbar_init(&bar_grant[q], 1);
    }
    for (int s = 0; s < KST; ++s) { mbar_init(&bar_kfull[s], 1); mbar_init(&bar_kempty[s], 1); }
    for (int s = 0; s < VST; ++s) { mbar_init(&bar_vfull[s], 1); mbar_init(&bar_vempty[s], 1); }
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
  // (the plan's scratch lies in the tiles: its generic accesses before the copies' writes)
  fence_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const uint32_t sbase = smem_u32(smem);
  auto sQ = [&](int q) { return sbase + C::Q_OFF + q * C::TILE_BYTES; };
  auto sK = [&](int st) { return sbase + C::K_OFF + st * C::TILE_BYTES; };
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

  if (warp >= C::SOFTMAX_WARPS) {
    regs_decrease<C::REGS_CONTROL>();
    if (warp == C::KQ_WARP) {
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
    } else if (warp == C::V_WARP) {
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
      const bool leader = lane == 0;
      int g = 0, j = 0;
      uint32_t pos = 0;
      while (next()) {
        const int n = seg.n;
        if (n == 0) { pos += 1; continue; }
        const int k0 = g % KST;
        for (int q = 0; q < NQ; ++q) {
          named_bar_sync(C::RELAY_BAR, 64);
          tc_fence_after();
          if (leader) {
            issue_qk<C>(tmem + C::s_col(q), sQ(q), sK(k0));
            tc_commit(&bar_s[q]);
            if (n == 1) tc_commit(&bar_qfree[q]);
          }
          __syncwarp();
        }
        if (leader) tc_commit(&bar_kempty[k0]);
        __syncwarp();
        for (int t = 0; t < n; ++t, ++g, ++pos) {
          const int vs = pos % VST, ks = (g + 1) % KST;
          const bool more = t + 1 < n;
          named_bar_sync(C::RELAY_BAR, 64);  // V_g (and K_{g+1}) are in shared memory
          for (int q = 0; q < NQ; ++q) {
            named_bar_sync(1 + q, 128 + 32);  // P_q(g) is in TMEM
            tc_fence_after();
            if (leader) {
              issue_pv<C, TERMS>(tmem + C::o_col(q), tmem + C::s_col(q), sV(vs), t > 0);
              if (more) {
                issue_qk<C>(tmem + C::s_col(q), sQ(q), sK(ks));
                tc_commit(&bar_s[q]);
                if (t + 2 == n) tc_commit(&bar_qfree[q]);
              } else {
                tc_commit(&bar_o[q]);
              }
            }
            __syncwarp();
          }
          if (leader) {
            tc_commit(&bar_vempty[vs]);
            if (more) tc_commit(&bar_kempty[ks]);
          }
          __syncwarp();
        }
        pos += 1;
        ++j;
      }
      if (j > 0 && leader) {
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
          if (ok && end < BLOCK_N) {
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
      float m = -FLT_MAX, l = 0.f;
      for (int t = 0; t < n; ++t, ++g) {
        if (live) live = __all_sync(0xffffffffu, wait_issuer(&bar_s[q], g & 1));
        if (!live) {
          named_bar_sync(1 + q, 128 + 32);  // every round is joined, whatever happens
          if (pending) release();
          continue;
        }
        tc_fence_after();
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
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : __fdividef(1.f, l);  // (NaN stays)
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

template <int D, int TERMS>
fa_status run(TilesArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  using C = TilesCfg<D>;
  auto* kernel = attend_tiles_kernel<D, TERMS>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return failed();
  const int ctas = host::sm_count();
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas, a.g.R, D), s) != cudaSuccess) return failed();
  a.part = partials_at(w, ctas, a.g.R, D);
  fa_status st;
  {
    host::KernelTimer t("attend_tiles", s);
    st = launch(kernel, ctas, C::THREADS, C::SMEM, s, q, k, v, a);
  }
  if (st == FA_OK) {
    const JoinArgs j = {a.part, a.O, a.LSE, ctas, 1, a.g.R, D, a.H, a.c.D, a.out_bf16, a.g.rep};
    st = launch_join_tall(j, s);
  }
  if (host::scratch_free(w, s) != cudaSuccess) st = failed();
  return st;
}

}  // namespace

fa_status launch_attend_tiles(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                              const fakv_cache& c, const fakv_tokens& p, cudaStream_t s) {
  if (host::sm_count() > TALL_CTAS) return FA_ERR_UNSUPPORTED;
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
  const uint64_t d = c.D, b2 = 2;
  CUtensorMap mq, mk, mv;
  // q as [HKV][T][rep][D], the pages as [page][head][token][D]
  const uint64_t qd[4] = {d, (uint64_t)rep, (uint64_t)p.T, (uint64_t)c.HKV};
  const uint64_t qs[3] = {(uint64_t)p.q_head * b2, (uint64_t)p.q_token * b2, (uint64_t)p.q_head * rep * b2};
  const uint32_t qb[4] = {64, (uint32_t)rep, (uint32_t)a.tpt, 1};
  const uint64_t kd[4] = {d, (uint64_t)c.page_size, (uint64_t)c.HKV, (uint64_t)c.num_pages};
  const uint64_t ks[3] = {(uint64_t)c.token_stride * b2, (uint64_t)c.head_stride * b2, (uint64_t)c.page_stride * b2};
  const uint32_t kb[4] = {64, (uint32_t)a.box, 1, 1};
  const long long plane = p.plane * c.plane_stride * 2;
  if (!host::encode_tiled_4d(&mq, q, qd, qs, qb) || !host::encode_tiled_4d(&mk, static_cast<const char*>(c.K) + plane, kd, ks, kb) ||
      !host::encode_tiled_4d(&mv, static_cast<const char*>(c.V) + plane, kd, ks, kb))
    return FA_ERR_UNSUPPORTED;
  if (a.out_bf16) return c.D <= 64 ? run<64, 1>(a, mq, mk, mv, s) : run<128, 1>(a, mq, mk, mv, s);
  return c.D <= 64 ? run<64, 2>(a, mq, mk, mv, s) : run<128, 2>(a, mq, mk, mv, s);
}

unsigned int read_and_clear_kv_status(cudaError_t* err) {
  unsigned int v = 0, zero = 0;
  *err = cudaMemcpyFromSymbol(&v, g_kv_status, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(zero));
  return v;
}

}  // namespace kv
}  // namespace fa
