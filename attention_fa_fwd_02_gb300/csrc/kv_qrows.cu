// kv_qrows.cu -- attention over the cache in 4 or 8 bits for few rows per sequence (decoding), and for
// fp32 queries: codes streamed once, made bf16 in registers, mma.sync.
//
// Workers, parts, copies and joins are those of kv_rows.cu. With s, z of a key's group g and codes
// c = centre + x (centre 8 or 128), its K and V are s x + z', z' = z + centre s, so that
//
//   scores  S = sum_g s_g (sum_{d in g} q_d x_d) + z'_g (sum_{d in g} q_d): codes are the exact bf16
//           operands of the products, a key's scales come after them, in fp32
//   O^T     O_d = sum_k (p_k s_k) x_kd + sum_k p_k z'_k: the scales enter the probabilities (two bf16
//           terms), the offsets are one more sum per row and group
//
// so nothing of the cache is rounded again. A code costs less than an instruction (kv_quant.cuh):
//   K  columns are what is summed over, in any order: a thread takes the 8 (4) columns of one
//      32-bit word of its key, and q's fragments are laid out to match
//   V  keys are summed over, two of each register: the halves of two keys' words are put side by side
//      first (one permute), so that every nibble pair is one column of two keys
#include <algorithm>
#include "kv_quant.cuh"
#include "kv_rows.cuh"

namespace fa {
namespace kv {
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
  int out_bf16;
  Partials part;
};

template <typename E, int BITS, int D, int NTR>
struct QRowsCfg {
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int TERMS = F32 ? 3 : 1;       // bf16 terms of q
  static constexpr int R = 8 * NTR;               // rows of an item
  static constexpr int CH = D * BITS / 128;       // 16-byte chunks of a key's codes
  static constexpr int NG = D / 64;               // groups of a key
  static constexpr int KS = D / 16;               // k16 steps of q
  static constexpr int GROUP = 32;                // keys of a step
  static constexpr int KT = GROUP / 16;
  static constexpr int CODES = GROUP * CH * 16;
  static constexpr int SLOT = CODES + GROUP * NG * 4;  // K (or V) of a step
  static constexpr bool Q_REGS = NTR == 1 && !F32;     // q's fragments stay in registers
  static constexpr int Q_BYTES = Q_REGS ? 0 : NTR * TERMS * (KS / 2) * 512;
  static constexpr int OS = D + 4;                // floats of a row of O in shared memory (bank spread)
  static constexpr int CTAS_PER_SM = Q_REGS ? 3 : 2;
  static constexpr int ROOM = CTAS_PER_SM == 3 ? 18432 : 28160;
  static constexpr int NS = std::min(12, (ROOM - Q_BYTES) / SLOT);
  static constexpr int WARP_BYTES = std::max({NS * SLOT + Q_BYTES, R * OS * 4, 16400});
  static constexpr int SMEM = WARPS * WARP_BYTES;
  static_assert(NS >= 2 && WARP_BYTES % 16 == 0 && SLOT % 16 == 0, "the ring");
  static_assert(SMEM >= 4 * 16385, "the plan's scratch");
  static constexpr int STATIC = (int)sizeof(PlanShared<NTHREADS, WARPS>) + WARPS * (R * 8 + 20);
  static_assert(CTAS_PER_SM * (SMEM + (STATIC + 1023) / 1024 * 1024 + 1024) <= 228 * 1024, "shared memory of the CTAs of an SM");
};

// x = sum of three bf16 terms
__device__ __forceinline__ void split3(float x, float (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= t[i];
  }
}

template <typename E, int BITS, int D, int NTR>
__global__ void __launch_bounds__(NTHREADS, QRowsCfg<E, BITS, D, NTR>::CTAS_PER_SM)
    qattend_rows_kernel(const __grid_constant__ QRowsArgs a) {
  using C = QRowsCfg<E, BITS, D, NTR>;
  constexpr int CH = C::CH, R = C::R, NS = C::NS, GROUP = C::GROUP, KT = C::KT, NG = C::NG, KS = C::KS;
  constexpr int TERMS = C::TERMS;
  constexpr bool CENTRED = C::F32;  // K's codes: centred before the product, or their constant taken off after it
  constexpr float CENTRE = BITS == 4 ? 8.f : 128.f;
  constexpr int WH = CH / 2;          // V words of a lane and key
  constexpr int J = BITS == 4 ? 4 : 2;  // output tiles of a word: columns j and j + J of each lane's
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ PlanShared<NTHREADS, WARPS> plan;
  __shared__ Ends<R> ends_sh;
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 3, oct = lane >> 2;  // mma fragments: columns 2 quad, 2 quad + 1; row oct
  const fakv_cache& c = a.c;
  const Geo& g = a.g;
  const int chunks = a.qc.chunks, ng = a.qc.groups;
  Seq seq;
  const Part part = find_part<NTHREADS, WARPS>(g, c, a.cu, a.slots, a.B, a.T, reinterpret_cast<int*>(smem), plan, seq);
  Walk walk(part, seq);
  const int worker = blockIdx.x * WARPS + warp;
  if (lane < 2) a.part.left[2 * worker + lane].flags = 0;
  if (lane == 0) ends_sh.item[warp] = make_int4(walk.p.b, walk.p.tile, walk.p.head, 2);
  uint8_t* const mine = smem + warp * C::WARP_BYTES;
  const uint32_t sq = ptx::smem_u32(mine);
  const uint32_t ring = sq + C::Q_BYTES;
  const long long v_minus_k = a.qc.V - a.qc.K;
  // V: lanes of the upper four octs read the odd key of a pair first (their banks are those that the
  // lower ones' even keys leave free), and put the halves together the other way round
  const int odd = oct >> 2;
  const uint32_t sel_lo = odd ? 0x1054u : 0x5410u, sel_hi = odd ? 0x3276u : 0x7632u;
  Seg seg = {};
  Finish fin;
  bool held = false;  // the worker's only item, not done whole: its result waits for the others'

  while (walk.next(g, c, a.cu, a.slots, a.T, seg)) {
    const Seq& s = seg.s;
    const Tile& x = seg.x;

    // ---- pages of the next 32 octets of keys, an octet per lane, and of the 32 after those:
    // look-ups are never waited for in the loop
    const int first = seg.k0 * GROUP;
    const int n = max(0, min(seg.k0 + seg.n, (x.hi + GROUP - 1) / GROUP) - seg.k0);  // steps
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

    // ---- copies of half-step j: K (j even) or V of step j / 2, octet by octet, each in a page
    const uint8_t* base[GROUP / 8];  // codes of the step's octets (null: zeros)
    const uint8_t* base_p = nullptr; // the lane's piece of the params
    uint32_t fill = ring;
    auto load = [&](int j) {
      if (j < 2 * n) {
        const bool is_v = j & 1;
        const long long v = is_v ? v_minus_k : 0;
        if (!is_v) {
          const int octet0 = (j >> 1) * (GROUP / 8);
          if ((octet0 & 31) == 0) {
            page = page_next;
            page_next = lookup(octet0 + 32 + lane);
          }
#pragma unroll
          for (int k = 0; k < GROUP / 8; ++k) {
            const int t = (first + (octet0 + k) * 8) & (c.page_size - 1);
            const int p = __shfl_sync(0xffffffffu, page, (octet0 + k) & 31);
            base[k] = p < 0 ? nullptr : a.qc.K + seg.head * a.qc.head + p * a.qc.page + t * chunks * 16;
          }
          const int k = lane / (2 * ng);  // (an octet's params are 2 ng pieces)
          const int t = (first + (octet0 + k) * 8) & (c.page_size - 1);
          const int p = __shfl_sync(0xffffffffu, page, (octet0 + min(k, GROUP / 8 - 1)) & 31);
          base_p = p < 0 ? nullptr
                         : a.qc.K + seg.head * a.qc.head + p * a.qc.page + a.qc.params + t * ng * 4 + (lane - k * 2 * ng) * 16;
        }
#pragma unroll
        for (int k = 0; k < GROUP / 8; ++k)
#pragma unroll
          for (int z = 0; z < (CH + 3) / 4; ++z) {
            const int piece = z * 32 + lane;
            if (piece < chunks * 8)
              cp16(fill + k * CH * 128 + piece * 16, base[k] ? base[k] + v + piece * 16 : a.qc.K, base[k] != nullptr);
          }
        if (lane < GROUP / 8 * 2 * ng) cp16(fill + C::CODES + lane * 16, base_p ? base_p + v : a.qc.K, base_p != nullptr);
        fill = fill + C::SLOT == ring + NS * C::SLOT ? ring : fill + C::SLOT;
      }
      cp_commit();
    };

    // ---- q: fragments of its rows (zeros behind the item's rows and the tensor's columns), and of
    // rows 8 nt + 2 quad + e the sums over each group: of q, and (not centred) of q times its codes' constants
    uint4 qr[C::Q_REGS ? KS / 2 : 1];
    float qs[NTR][NG][2], qb[NTR][NG][2];
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) {
      const int r = nt * 8 + oct;
      const int rho = x.rho0 + min(r, x.rows - 1), token = g.rep.of(rho);
      const E* const src = static_cast<const E*>(a.q) + (s.row0 + token) * a.q_token +
                           (seg.head * g.rep.d + rho - token * g.rep.d) * a.q_head;
      float sum[NG], bias[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) sum[i] = bias[i] = 0.f;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {  // two k16 steps: 4 bits: 8 columns of block i; 8 bits: 4 of chunks 2 i and 2 i + 1
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // four columns each
          const int col = BITS == 4 ? i * 32 + quad * 8 + e * 4 : (2 * i + e) * 16 + quad * 4;
          if (r < x.rows && col < c.D) {
            if constexpr (C::F32) {
              const float4 v = *reinterpret_cast<const float4*>(src + col);
              y[4 * e] = v.x; y[4 * e + 1] = v.y; y[4 * e + 2] = v.z; y[4 * e + 3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src + col);
              y[4 * e] = __uint_as_float(v.x << 16); y[4 * e + 1] = __uint_as_float(v.x & 0xffff0000u);
              y[4 * e + 2] = __uint_as_float(v.y << 16); y[4 * e + 3] = __uint_as_float(v.y & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[i / 2] += y[e];
          // 4 bits: column e is nibble e, of pair e % 4; 8 bits: byte e % 4's nibbles, of pairs 2 (e % 2) and + 1
          bias[i / 2] += y[e] * (BITS == 4 ? q_bias(e & 3) : 256.f + q_bias(2 * (e & 1)));
        }
        // pairs: 4 bits (0, 4), (1, 5), (2, 6), (3, 7); 8 bits (0, 2), (1, 3) of each chunk
        constexpr int A0[4] = {0, 1, BITS == 4 ? 2 : 4, BITS == 4 ? 3 : 5}, GAP = BITS == 4 ? 4 : 2;
        if constexpr (C::Q_REGS) {
          qr[i] = make_uint4(bf2(y[A0[0]], y[A0[0] + GAP]), bf2(y[A0[1]], y[A0[1] + GAP]), bf2(y[A0[2]], y[A0[2] + GAP]),
                             bf2(y[A0[3]], y[A0[3] + GAP]));
        } else {
          float t[8][3];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (C::F32) split3(y[e], t[e]);
            else t[e][0] = y[e];
          }
#pragma unroll
          for (int m = 0; m < TERMS; ++m)
            ptx::st_shared_v4(sq + ((nt * TERMS + m) * (KS / 2) + i) * 512 + lane * 16, bf2(t[A0[0]][m], t[A0[0] + GAP][m]),
                              bf2(t[A0[1]][m], t[A0[1] + GAP][m]), bf2(t[A0[2]][m], t[A0[2] + GAP][m]),
                              bf2(t[A0[3]][m], t[A0[3] + GAP][m]));
        }
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        bias[i] += __shfl_xor_sync(0xffffffffu, bias[i], 1);
        bias[i] += __shfl_xor_sync(0xffffffffu, bias[i], 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qs[nt][i][e] = __shfl_sync(0xffffffffu, sum[i], (2 * quad + e) * 4);
          qb[nt][i][e] = __shfl_sync(0xffffffffu, bias[i], (2 * quad + e) * 4);
        }
      }
    }
    __syncwarp();

    // rows 8 nt + 2 quad + e; o: columns (h's) base + j, base + j + J
    float m[NTR][2], l[NTR][2], o[WH][J][NTR][4], oz[NTR][NG][2];
#pragma unroll
    for (int nt = 0; nt < NTR; ++nt) {
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) oz[nt][i][0] = oz[nt][i][1] = 0.f;
#pragma unroll
      for (int h = 0; h < WH; ++h)
#pragma unroll
        for (int j = 0; j < J; ++j) o[h][j][nt][0] = o[h][j][nt][1] = o[h][j][nt][2] = o[h][j][nt][3] = 0.f;
    }
    // keys that every row sees need no mask
    int in_lo, in_hi;
    {
      const int pa = s.len - s.n + g.rep.of(x.rho0), pb = s.len - s.n + g.rep.of(x.rho0 + x.rows - 1);
      in_hi = g.causal ? min(pa, s.len - 1) : s.len - 1;
      in_lo = g.window > 0 ? pb - g.window + 1 : 0;
    }

    // Half-steps K_0, V_0, K_1, ...: a slot is filled again as soon as it is read, NS half-steps
    // ahead. The first NS rounds only load.
    uint32_t use = ring;
    float sc[KT][NTR][4];  // scores, then probabilities: keys 16 kt + oct (+ 8), rows 8 nt + 2 quad + e
#pragma unroll 1
    for (int j = -NS; j < 2 * n; ++j) {
      if (j >= 0) {
        cp_wait<NS - 1>();
        __syncwarp();
        const int j0 = first + (j >> 1) * GROUP;
        const bool edge = j0 < in_lo || j0 + GROUP - 1 > in_hi;
        // s and z' of key 16 kt + 8 e + oct, group i
        auto params = [&](int kt, int e, float (&ps)[NG], float (&pz)[NG], bool centred) {
          const uint32_t at = use + C::CODES + (kt * 16 + e * 8 + oct) * ng * 4;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const uint32_t p = lds32(at + (i && ng > 1 ? 4 : 0));
            ps[i] = q_scale(p);
            pz[i] = centred ? fmaf(ps[i], CENTRE, q_offset(p)) : q_offset(p);
          }
        };
        if ((j & 1) == 0) {
          // -------- scores of step j / 2
          float acc[NG][KT][NTR][4];
#pragma unroll
          for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][kt][nt][e] = CENTRED ? 0.f : -qb[nt][i][e & 1];
#pragma unroll
          for (int w = 0; w < CH; ++w) {
            if (w >= chunks) break;
            uint32_t word[KT][2];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int e = 0; e < 2; ++e) word[kt][e] = lds32(use + ((kt * 2 + e) * CH + w) * 128 + lane * 4);
            constexpr int PER = BITS == 4 ? 2 : 1;  // k16 steps of q for a chunk
#pragma unroll
            for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
              for (int t = TERMS - 1; t >= 0; --t) {
                const int step = w * PER;
                uint4 v;
                if constexpr (C::Q_REGS) v = qr[step / 2];
                else {
                  const float4 f = ptx::ld_shared_v4(sq + ((nt * TERMS + t) * (KS / 2) + step / 2) * 512 + lane * 16);
                  v = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
                }
                const uint32_t b0 = step & 1 ? v.z : v.x, b1 = step & 1 ? v.w : v.y;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                  const uint32_t lo = word[kt][0], hi = word[kt][1];
                  float(&d)[4] = acc[BITS == 4 ? w / 2 : w / 4][kt][nt];
                  if constexpr (BITS == 4) {
                    uint32_t f0[4], f1[4];
                    if constexpr (CENTRED) {
                      f0[0] = q_centred4<0>(lo); f0[1] = q_centred4<0>(hi); f0[2] = q_centred4<1>(lo); f0[3] = q_centred4<1>(hi);
                      f1[0] = q_centred4<2>(lo); f1[1] = q_centred4<2>(hi); f1[2] = q_centred4<3>(lo); f1[3] = q_centred4<3>(hi);
                    } else {
                      f0[0] = q_pair<0>(lo); f0[1] = q_pair<0>(hi); f0[2] = q_pair<1>(lo); f0[3] = q_pair<1>(hi);
                      f1[0] = q_pair<2>(lo); f1[1] = q_pair<2>(hi); f1[2] = q_pair<3>(lo); f1[3] = q_pair<3>(hi);
                    }
                    mma_bf16(d, f0, v.x, v.y);
                    mma_bf16(d, f1, v.z, v.w);
                  } else if constexpr (CENTRED) {
                    const uint32_t f[4] = {q_centred8<0>(lo), q_centred8<0>(hi), q_centred8<1>(lo), q_centred8<1>(hi)};
                    mma_bf16(d, f, b0, b1);
                  } else {
                    const uint32_t f0[4] = {q_pair<0>(lo), q_pair<0>(hi), q_pair<2>(lo), q_pair<2>(hi)};
                    const uint32_t f1[4] = {q_pair16<1>(lo), q_pair16<1>(hi), q_pair16<3>(lo), q_pair16<3>(hi)};
                    mma_bf16(d, f0, b0, b1);
                    mma_bf16(d, f1, b0, b1);
                  }
                }
              }
          }
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float ps[NG], pz[NG];
              params(kt, z, ps, pz, CENTRED);
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float v = pz[0] * qs[nt][0][e];
#pragma unroll
                  for (int i = 0; i < NG; ++i) {
                    if (i > 0) v = fmaf(pz[i], qs[nt][i][e], v);
                    v = fmaf(ps[i], acc[i][kt][nt][2 * z + e], v);
                  }
                  sc[kt][nt][2 * z + e] = v;
                }
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
                for (int i = 0; i < NG; ++i) oz[nt][i][e] *= f;
#pragma unroll
                for (int h = 0; h < WH; ++h)
#pragma unroll
                  for (int t = 0; t < J; ++t) {
                    o[h][t][nt][e] *= f;
                    o[h][t][nt][e + 2] *= f;
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
        } else {
          // -------- O^T += V^T (s P)^T, and the offsets' sums
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            uint32_t ph[NG][NTR][2], pl[NG][NTR][2];  // keys low, high
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float ps[NG], pz[NG];
              params(kt, z, ps, pz, true);
#pragma unroll
              for (int nt = 0; nt < NTR; ++nt)
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                  const float p0 = sc[kt][nt][2 * z], p1 = sc[kt][nt][2 * z + 1];
                  float s0 = p0 * ps[i], s1 = p1 * ps[i], z0 = p0 * pz[i], z1 = p1 * pz[i];
                  if (edge) {  // a key that a row does not see may be anything
                    if (p0 == 0.f) s0 = z0 = 0.f;
                    if (p1 == 0.f) s1 = z1 = 0.f;
                  }
                  oz[nt][i][0] += z0;
                  oz[nt][i][1] += z1;
                  const uint32_t hi = bf2(s0, s1);
                  ph[i][nt][z] = transpose8(hi);
                  pl[i][nt][z] = transpose8(bf2(s0 - __uint_as_float(hi << 16), s1 - __uint_as_float(hi & 0xffff0000u)));
                }
            }
#pragma unroll
            for (int h = 0; h < WH; ++h) {
              if (2 * h >= chunks) break;
              const int i = BITS == 4 ? h : h / 2;  // the words' group
              uint32_t half[2][2];  // keys low, high: the words' low and high halves, of two keys
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // (an odd number of chunks: the upper octs read the last one again, for columns that do not exist)
                const uint32_t at = use + ((kt * 2 + z) * CH + min(2 * h + odd, chunks - 1)) * 128 + quad * 32 + (oct & 3) * 4;
                const uint32_t p = lds32(at + odd * 16), q = lds32(at + 16 - odd * 16);
                half[z][0] = __byte_perm(p, q, sel_lo);
                half[z][1] = __byte_perm(p, q, sel_hi);
              }
              auto tile = [&](auto jj) {
                constexpr int t = decltype(jj)::value;
                const uint32_t va[4] = {q_centred<BITS, t>(half[0][0]), q_centred<BITS, t>(half[0][1]),
                                        q_centred<BITS, t>(half[1][0]), q_centred<BITS, t>(half[1][1])};
#pragma unroll
                for (int nt = 0; nt < NTR; ++nt) {
                  mma_bf16(o[h][t][nt], va, pl[i < NG ? i : 0][nt][0], pl[i < NG ? i : 0][nt][1]);
                  mma_bf16(o[h][t][nt], va, ph[i < NG ? i : 0][nt][0], ph[i < NG ? i : 0][nt][1]);
                }
              };
              tile(std::integral_constant<int, 0>());
              tile(std::integral_constant<int, 1>());
              if constexpr (BITS == 4) {
                tile(std::integral_constant<int, 2>());
                tile(std::integral_constant<int, 3>());
              }
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
        auto over_keys = [](float v) {
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          return v + __shfl_xor_sync(0xffffffffu, v, 16);
        };
        const float v = over_keys(l[nt][e]);
        float z[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) z[i] = over_keys(oz[nt][i][e]);
        const int r = nt * 8 + quad * 2 + e;
        if (oct == 0) ends_sh.ml[warp][r] = make_float2(m[nt][e], v);
        float* const to = reinterpret_cast<float*>(mine) + r * C::OS + oct * 2 * J;
#pragma unroll
        for (int h = 0; h < WH; ++h)
#pragma unroll
          for (int t = 0; t < J; ++t) {
            const float zh = z[(BITS == 4 ? h : h / 2) % NG];
            to[h * 16 * J + t] = o[h][t][nt][e] + zh;
            to[h * 16 * J + t + J] = o[h][t][nt][e + 2] + zh;
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

template <typename E, int BITS, int D, int NTR>
fa_status run(QRowsArgs& a, cudaStream_t s) {
  using C = QRowsCfg<E, BITS, D, NTR>;
  auto* kernel = qattend_rows_kernel<E, BITS, D, NTR>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, C::SMEM, done)) return failed();
  const int ctas = host::sm_count() * C::CTAS_PER_SM;
  void* w = nullptr;
  if (host::scratch_alloc(&w, partials_bytes(ctas * WARPS, C::R, D), s) != cudaSuccess) return failed();
  a.part = partials_at(w, ctas * WARPS, C::R, D);
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

template <typename E, int BITS>
fa_status pick(QRowsArgs& a, long long rows, cudaStream_t s) {
  if (a.c.D <= 64) return rows <= 8 ? run<E, BITS, 64, 1>(a, s) : run<E, BITS, 64, 2>(a, s);
  return rows <= 8 ? run<E, BITS, 128, 1>(a, s) : run<E, BITS, 128, 2>(a, s);
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
  a.out_bf16 = p.out_dtype == FA_BF16;
  // Items of 8 or 16 rows: what a sequence's rows fit on average
  const long long rows = ((long long)p.T * rep + p.B - 1) / p.B;
  if (c.dtype == FA_BF16) return qc.bits == 4 ? pick<__nv_bfloat16, 4>(a, rows, s) : pick<__nv_bfloat16, 8>(a, rows, s);
  return qc.bits == 4 ? pick<float, 4>(a, rows, s) : pick<float, 8>(a, rows, s);
}

}  // namespace kv
}  // namespace fa
