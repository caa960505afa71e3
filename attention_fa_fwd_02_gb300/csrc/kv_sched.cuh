// kv_sched.cuh -- how attention over the paged cache is shared out among the CTAs.
//
// An item is one tile of `R` rows of one sequence and kv head (row r of a sequence: token
// r / rep, query head head * rep + r % rep, so the heads that read one kv head share its
// keys). It costs the units of `U` keys that its rows may see, at least one. All items in
// order (sequence, tile, head), the units of an item in key order, form one line, which is
// cut into equal parts, one per CTA, whatever the lengths are: a long sequence is spread
// over many CTAs, and a CTA may take many short ones. Every CTA finds its own part from
// the lengths (on the device: the host knows none). A part begins or ends inside an item at
// most once each, so a CTA leaves at most two partial results (output and softmax
// statistics), in slots of its own; attend_join_kernel puts an item's parts together in key
// order. Cuts depend on the lengths alone, so results do too.
#pragma once
#include "kv_common.cuh"

namespace fa {
namespace kv {

struct Geo {
  int rep, R, U;        // heads per kv head; rows per item; keys per unit
  int causal, window;
};

struct Tile {
  int rows;         // rows of the item
  int rho0;         // its first row within the sequence
  int lo, hi;       // keys [lo, hi) that any of its rows sees (empty: lo == hi == 0)
  int u0, units;    // units of keys
  int cost;
};

__device__ __forceinline__ Tile tile_of(const Geo& g, const Seq& s, int t) {
  Tile x;
  x.rho0 = t * g.R;
  x.rows = min(g.R, s.n * g.rep - x.rho0);
  const int i0 = x.rho0 / g.rep, i1 = (x.rho0 + x.rows - 1) / g.rep;
  const int p0 = s.len - s.n + i0, p1 = s.len - s.n + i1;
  x.hi = g.causal ? min(s.len, p1 + 1) : s.len;
  x.lo = g.window > 0 ? max(0, p0 - g.window + 1) : 0;
  if (x.hi <= x.lo) x.lo = x.hi = 0;
  x.u0 = x.lo / g.U;
  x.units = (x.hi + g.U - 1) / g.U - x.u0;
  x.cost = max(1, x.units);
  return x;
}

__device__ __forceinline__ int tiles_of(const Geo& g, int n) { return (n * g.rep + g.R - 1) / g.R; }

template <int NT>
__device__ __forceinline__ long long scan_ll(long long x, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += v;
  }
  if (lane == 31) warp_sums[w] = y;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    if (k < w) before += warp_sums[k];
    all += warp_sums[k];
  }
  *total = all;
  __syncthreads();
  return before + y - x;
}

struct Part {      // a CTA's part of the line
  int b, tile, head, unit;
  long long units; // 0: none
};

struct PlanShared {
  long long sums[16];
  Part part;
};

// The part of CTA `cta` of `ctas`, by a block of NT threads. `first`: shared scratch of
// B + 1 ints (used within the call only).
template <int NT>
__device__ __forceinline__ Part find_part(const Geo& g, const fakv_cache& c, const int* cu,
                                          const int* slots, int B, int T, int* first,
                                          PlanShared& sh, int cta, int ctas) {
  const int tid = threadIdx.x;
  // tiles of the sequences before each
  const int per = (B + NT - 1) / NT;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long n = 0, total;
  for (int b = b0; b < b1; ++b) n += tiles_of(g, load_seq(c, cu, slots, b, T).n);
  long long at = scan_ll<NT>(n, sh.sums, &total);
  const int tiles = (int)total;
  for (int b = b0; b < b1; ++b) {
    first[b] = (int)at;
    at += tiles_of(g, load_seq(c, cu, slots, b, T).n);
  }
  if (tid == 0) { first[B] = tiles; sh.part.units = 0; }
  __syncthreads();
  // cost of the tiles before each thread's
  const int q = (tiles + NT - 1) / NT;
  const int t0 = min(tiles, tid * q), t1 = min(tiles, t0 + q);
  int lo = 0;
  if (t0 < t1) {
    int hi = B;  // the last b with first[b] <= t0 has a tile t0 (empty sequences share the next one's)
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= t0) lo = mid; else hi = mid;
    }
  }
  long long cost = 0;
  {
    int b = lo;
    Seq s;
    for (int t = t0; t < t1; ++t) {
      if (t == t0 || t >= first[b + 1]) {
        while (t >= first[b + 1]) ++b;
        s = load_seq(c, cu, slots, b, T);
      }
      cost += tile_of(g, s, t - first[b]).cost;
    }
  }
  long long before = scan_ll<NT>(cost, sh.sums, &total);
  total *= c.HKV;
  const int used = (int)min((long long)ctas, total);
  if (cta < used) {
    auto cut = [&](int k) { return total / used * k + total % used * k / used; };
    const long long x0 = cut(cta), x1 = cut(cta + 1);
    if (t0 < t1 && before * c.HKV <= x0 && x0 < (before + cost) * c.HKV) {
      int b = lo;
      Seq s;
      long long at = before * c.HKV;
      for (int t = t0; t < t1; ++t) {
        if (t == t0 || t >= first[b + 1]) {
          while (t >= first[b + 1]) ++b;
          s = load_seq(c, cu, slots, b, T);
        }
        const int k = tile_of(g, s, t - first[b]).cost;
        if (x0 < at + (long long)k * c.HKV) {
          const int off = (int)(x0 - at);
          sh.part = {b, t - first[b], off / k, off % k, x1 - x0};
          break;
        }
        at += (long long)k * c.HKV;
      }
    }
  }
  __syncthreads();
  return sh.part;
}

// A CTA's way along its part, an item (or what of it lies in the part) at a time.
struct Seg {
  Seq s;
  Tile x;
  int head;
  int k0, n;          // units [k0, k0 + n) of keys (n = 0: an item that sees none)
  bool starts, ends;  // the item begins / ends here
  int slot;           // of a partial result: 0 or 1
};

struct Walk {
  int b, tile, head, unit;
  long long left;
  Seq s;
  bool moved;
  __device__ __forceinline__ Walk(const Part& p) : b(p.b), tile(p.tile), head(p.head), unit(p.unit), left(p.units), moved(false) {}
  __device__ __forceinline__ bool next(const Geo& g, const fakv_cache& c, const int* cu, const int* slots, int T, Seg& o) {
    if (left <= 0) return false;
    if (!moved) s = load_seq(c, cu, slots, b, T);
    else if (unit == 0 && head == 0) {
      while (tile * g.R >= s.n * g.rep) {  // the next sequence with rows
        tile = 0;
        s = load_seq(c, cu, slots, ++b, T);
      }
    }
    o.s = s;
    o.x = tile_of(g, s, tile);
    o.head = head;
    o.slot = moved ? 1 : 0;
    const int take = (int)min((long long)(o.x.cost - unit), left);
    o.k0 = o.x.u0 + unit;
    o.n = min(take, o.x.units - unit);
    o.starts = unit == 0;
    o.ends = unit + take == o.x.cost;
    left -= take;
    unit += take;
    moved = true;
    if (o.ends) {
      unit = 0;
      if (++head == c.HKV) { head = 0; ++tile; }
    }
    return true;
  }
};

// What a CTA left of an item that it did not do whole: slot 2 * cta (the item its part
// begins in) or 2 * cta + 1 (the one it ends in).
enum { PART_VALID = 1, PART_STARTS = 2, PART_ENDS = 4 };
struct Left {
  int flags, row0, rho0, rows, head, pad[3];
};

// Partial results: O [slots][R][D] not normalised, and per row the maximum m (log2 units)
// its exponentials were taken against and their sum l.
struct Partials {
  Left* left;
  float* O;
  float2* ml;
};

inline size_t partials_bytes(int ctas, int R, int D) {
  return (size_t)ctas * 2 * (sizeof(Left) + (size_t)R * (D + 2) * 4);
}
inline Partials partials_at(void* p, int ctas, int R, int D) {
  Partials x;
  x.left = static_cast<Left*>(p);
  x.O = reinterpret_cast<float*>(x.left + 2 * ctas);
  x.ml = reinterpret_cast<float2*>(x.O + (size_t)2 * ctas * R * D);
  return x;
}

struct JoinArgs {
  Partials part;
  void* O;
  float* LSE;
  int ctas, R, D;  // D: columns of a partial row
  int H, rep, Dv, out_bf16;
};
fa_status launch_join(const JoinArgs& a, cudaStream_t s);

}  // namespace kv
}  // namespace fa
