// kv_sched.cuh -- how attention over the paged cache is shared out among the CTAs.
//
// An item is one tile of `R` rows of one sequence and kv head (row r of a sequence: token
// r / rep, query head head * rep + r % rep, so the heads that read one kv head share its
// keys). Its keys come in units of `U`. All items in order (sequence, tile, head), the units
// of an item in key order, form one line, on which an item also weighs `start` units more
// (what beginning an item costs a worker). The line is cut into equal parts, one per worker (a
// CTA, or a warp), whatever the lengths are: a long sequence is spread over many workers,
// and a worker may take many short ones; a cut that falls into an item of at most `snap` units
// (or an eighth of a part) moves to its nearer end. Every CTA finds its workers' parts from
// the lengths (on the device: the host knows none). A part begins or ends inside an item at
// most once each, so a worker leaves at most two partial results (output and softmax
// statistics), in slots of its own; the join puts an item's parts together in key order. Cuts
// depend on the lengths alone, so results do too.
#pragma once
#include "kv_common.cuh"

namespace fa {
namespace kv {

// n / d for 0 <= n < 2^31 by a product (d fixed for a launch; Granlund and Montgomery's
// division by invariant integers): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, t = high word of m n, it is (t + (n - t) / 2) / 2^(s - 1).
struct Div {
  unsigned m;
  int d, s1, s2;
  __device__ __forceinline__ int of(int n) const {
    const unsigned t = __umulhi(m, (unsigned)n);
    return (int)((t + (((unsigned)n - t) >> s1)) >> s2);
  }
};
inline Div div_by(int d) {
  const int s = log2_of(d);
  return {(unsigned)(((1ull << 32) * ((1ull << s) - d)) / d + 1), d, s < 1 ? s : 1, s > 1 ? s - 1 : 0};
}

struct Geo {
  Div rep;              // query heads per kv head
  int R;                // rows per item
  int u_shift;          // log2 of the keys of a unit
  int start, snap;
  int causal, window;
};

struct Tile {
  int rows;         // rows of the item
  int rho0;         // its first row within the sequence
  int lo, hi;       // keys [lo, hi) that any of its rows sees (empty: lo == hi == 0)
  int u0, units;    // units of keys
};

__device__ __forceinline__ Tile tile_of(const Geo& g, const Seq& s, int t) {
  Tile x;
  x.rho0 = t * g.R;
  x.rows = min(g.R, s.n * g.rep.d - x.rho0);
  const int p0 = s.len - s.n + g.rep.of(x.rho0), p1 = s.len - s.n + g.rep.of(x.rho0 + x.rows - 1);
  x.hi = g.causal ? min(s.len, p1 + 1) : s.len;
  x.lo = g.window > 0 ? max(0, p0 - g.window + 1) : 0;
  if (x.hi <= x.lo) x.lo = x.hi = 0;
  x.u0 = x.lo >> g.u_shift;
  x.units = ((x.hi + (1 << g.u_shift) - 1) >> g.u_shift) - x.u0;
  return x;
}

// tiles of a sequence of n new tokens (a division: R is no power of two)
__device__ __forceinline__ int tiles_of(const Geo& g, int n) { return (max(0, n) * g.rep.d + g.R - 1) / g.R; }

// Exclusive prefix sums of two values over the block (NT threads), and their totals.
template <int NT>
__device__ __forceinline__ void scan2(int& n, long long& w, int* n_total, long long* w_total, int* n_sums,
                                      long long* w_sums) {
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  int x = n;
  long long y = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, d);
    const long long v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) { x += u; y += v; }
  }
  if (lane == 31) { n_sums[k] = x; w_sums[k] = y; }
  __syncthreads();
  n = x - n;
  w = y - w;
  *n_total = 0;
  *w_total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const int u = n_sums[i];
    const long long v = w_sums[i];
    if (i < k) { n += u; w += v; }
    *n_total += u;
    *w_total += v;
  }
  __syncthreads();
}

// A worker's part: from unit `unit` of item (tile, head) up to (not including) unit
// `end_unit` of item (end_tile, end_head). Tiles are numbered over all sequences; `first`: that
// of the sequence b's first tile.
struct Part {
  int b, first, tile, head, unit;
  int end_tile, end_head, end_unit;
  int ender;  // the worker that ends the item (end_tile, end_head)
};

template <int NT, int PER>
struct PlanShared {
  long long w_sums[NT / 32];
  int n_sums[NT / 32];
  struct {       // where a cut falls: among the tiles [t0, ...) whose weights begin at `before`
    int b, t0;
    long long before;
  } own[PER + 1];
};

// Where worker k's part begins on a line of weight `total`: equal parts, the first `more` of
// them one longer.
struct Cuts {
  long long total, workers, len, more;
  __device__ __forceinline__ Cuts(long long total_, long long most) : total(total_), workers(min(most, total_)) {
    len = workers == 0 ? 0 : div(total, workers);
    more = total - len * workers;
  }
  static __device__ __forceinline__ long long div(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
  }
  __device__ __forceinline__ long long at(long long k) const {
    k = min(k, workers);
    return len * k + min(k, more);
  }
  __device__ __forceinline__ int worker_of(long long x) const {  // the inverse
    const long long bent = more * (len + 1);
    return (int)(x < bent ? div(x, len + 1) : more + div(x - bent, len));
  }
};

// A cut: the unit of an item that a part begins with, and the worker that ends the item
struct Cut {
  int tile, head, unit, ender;
};
// of a cut `off` into the weight of tile `tile` (all heads), each head of which has `cost` units
__device__ __forceinline__ Cut cut_in(const Geo& g, const Cuts& cuts, int HKV, int tile, int cost, long long x,
                                      long long off) {
  const int one = cost + g.start;
  Cut r;
  r.tile = tile;
  r.head = (int)Cuts::div(off, one);
  r.unit = (int)(off - (long long)r.head * one);
  r.ender = 0;
  if (cost <= max((long long)g.snap, cuts.len / 8)) {
    r.head += 2 * r.unit >= one;
    r.unit = 0;
    if (r.head == HKV) { r.head = 0; ++r.tile; }
  } else {
    r.ender = cuts.worker_of(x - r.unit + one - 1);  // who has the item's last unit
    r.unit = max(0, r.unit - g.start);
  }
  return r;
}

// The part of the caller's warp, worker PER * blockIdx.x + w (PER == 1: every warp gets the
// CTA's part), and its first sequence, found by a block of NT threads. `first`: shared
// scratch of B + 1 ints (used within the call only). All of it is latency, before the first
// key is asked for: up to 128 sequences of a few tiles each, as in decoding, or 32 of many, a
// warp finds its part by itself without meeting the others (one sequence: 3000 clocks instead of 6400
// by the block; 64: 5800 instead of 6900).
template <int NT, int PER>
__device__ __forceinline__ Part find_part(const Geo& g, const fakv_cache& c, const int* cu,
                                          const int* slots, int B, int T, int* first,
                                          PlanShared<NT, PER>& sh, Seq& seq) {
  constexpr int FEW = 4, ALONE = 128;
  const int tid = threadIdx.x, lane = tid & 31;
  const long long most = (long long)gridDim.x * PER;
  // every warp looks for its own two cuts: one in lane 0, the other in the rest
  const long long worker = (long long)blockIdx.x * PER + (PER == 1 ? 0 : tid / 32) + (lane > 0);
  Part p;
  Seq s = {};
  int b = B, f = 0;  // of lane 0: the part's first sequence, the number of its first tile
  Cut cut;
  const int per_lane = (B + 31) / 32;
  bool alone = per_lane <= ALONE / 32;
  int n = 0;                // tiles of the lane's sequences
  long long mine = 0;       // a lane's weight
  int lane_b = lane * per_lane, lane_t = 0;  // the sequence and the tile of it that a lane begins with
  bool falls = false;       // cu decreases
  if (alone) {
    bool many = false;
#pragma unroll 1
    for (int i = 0; i < per_lane; ++i) {
      const int at = lane * per_lane + i;
      if (at >= B) break;
      s = load_seq(c, cu, slots, at, T);
      falls |= s.n < 0;
      const int tiles = tiles_of(g, s.n);
      n += tiles;
      many |= tiles > FEW;
#pragma unroll 1
      for (int t = 0; t < tiles && !many; ++t) mine += max(1, tile_of(g, s, t).units) + g.start;
    }
    falls = __any_sync(0xffffffffu, falls);
    many = __any_sync(0xffffffffu, many) && !falls;
    alone = !many || per_lane == 1;
    if (falls) n = 0, mine = 0;
    if (alone && many) {
      // few sequences of many tiles: the tiles shared out evenly instead
      int t_end = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, t_end, d);
        if (lane >= d) t_end += u;
      }
      const int tiles = __shfl_sync(0xffffffffu, t_end, 31), q = (tiles + 31) / 32;
      int t = lane * q, at = 0;  // a tile, its sequence
      for (int k = 0; k < B; ++k) at += __shfl_sync(0xffffffffu, t_end, k) <= t;
      lane_b = at;
      lane_t = t - __shfl_sync(0xffffffffu, t_end - n, min(at, 31));
      mine = 0;
#pragma unroll 1
      for (int i = 0; i < q; ++i, ++t) {
        for (int k = 0; k <= B; ++k) {  // (every lane takes part in every exchange)
          const int end = __shfl_sync(0xffffffffu, t_end, min(at, 31));
          const bool on = t < tiles && end <= t;
          at += on;
          if (!__any_sync(0xffffffffu, on)) break;
        }
        const int from = min(at, 31);
        Seq o;
        o.slot = 0;
        o.len = __shfl_sync(0xffffffffu, s.len, from);
        o.row0 = 0;
        o.n = __shfl_sync(0xffffffffu, s.n, from);
        const int t_first = __shfl_sync(0xffffffffu, t_end - n, from);
        if (t < tiles) mine += max(1, tile_of(g, o, t - t_first).units) + g.start;
      }
      n = max(0, min(q, tiles - lane * q));  // tiles of the lane
    }
  }
  if (alone) {
    mine *= c.HKV;
    long long w_end = mine;
    int t_end = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t_end, d);
      const long long v = __shfl_up_sync(0xffffffffu, w_end, d);
      if (lane >= d) { t_end += u; w_end += v; }
    }
    const Cuts cuts(__shfl_sync(0xffffffffu, w_end, 31), most);
    const int tiles = __shfl_sync(0xffffffffu, t_end, 31);
    const long long x = cuts.at(worker);
    // the lane whose tiles each cut falls into: how many end at or before it
    const long long x0 = __shfl_sync(0xffffffffu, x, 0), x1 = __shfl_sync(0xffffffffu, x, 1);
    const int l0 = __popc(__ballot_sync(0xffffffffu, w_end <= x0)), l1 = __popc(__ballot_sync(0xffffffffu, w_end <= x1));
    const int from = min(31, lane > 0 ? l1 : l0);
    long long at = __shfl_sync(0xffffffffu, w_end - mine, from);
    int t = __shfl_sync(0xffffffffu, lane_t, from);  // tile of sequence b
    f = __shfl_sync(0xffffffffu, t_end - n, from) - t;
    b = __shfl_sync(0xffffffffu, lane_b, from);
    cut = {tiles, 0, 0, 0};
    if (x < cuts.total) {
      s = load_seq(c, cu, slots, b, T);
      int of = tiles_of(g, s.n);
#pragma unroll 1
      for (;; ++t) {
        while (t >= of) {
          f += of;
          t = 0;
          s = load_seq(c, cu, slots, ++b, T);
          of = tiles_of(g, s.n);
        }
        const int cost = max(1, tile_of(g, s, t).units);
        const long long span = (long long)(cost + g.start) * c.HKV;
        if (x < at + span) {
          cut = cut_in(g, cuts, c.HKV, f + t, cost, x, x - at);
          break;
        }
        at += span;
      }
    } else {
      f = tiles;
      b = B;
    }
  } else {
    // tiles of the sequences before each
    const int per = (B + NT - 1) / NT;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int at = 0, tiles;
    long long total, none = 0;
#pragma unroll 1
    for (b = b0; b < b1; ++b) {
      const int rows = load_seq(c, cu, slots, b, T).n;
      falls |= rows < 0;
      at += tiles_of(g, rows);
    }
    falls = __syncthreads_or(falls);
    scan2<NT>(at, none, &tiles, &total, sh.n_sums, sh.w_sums);
    if (falls) tiles = 0;
#pragma unroll 1
    for (b = b0; b < b1; ++b) {
      first[b] = at;
      if (b + 1 < b1) at += tiles_of(g, load_seq(c, cu, slots, b, T).n);
    }
    if (tid == 0) first[B] = tiles;
    __syncthreads();
    // the tiles shared out evenly: weights of those before each thread's
    const int q = (tiles + NT - 1) / NT;
    const int t0 = min(tiles, tid * q), t1 = min(tiles, t0 + q);
    b = 0;
    for (int hi = B; t0 < t1 && hi - b > 1;) {
      // the last b with first[b] <= t0 has a tile t0 (empty sequences share the next one's)
      const int mid = (b + hi) / 2;
      if (first[mid] <= t0) b = mid; else hi = mid;
    }
    const int b_t0 = b;
    bool have = false;
    auto units_of = [&](int t) {  // (tiles in order)
      if (!have || t >= first[b + 1]) {
        while (t >= first[b + 1]) ++b;
        s = load_seq(c, cu, slots, b, T);
        have = true;
      }
      return max(1, tile_of(g, s, t - first[b]).units);
    };
    long long mine = 0;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) mine += units_of(t) + g.start;
    mine *= c.HKV;
    long long before = mine;
    int zero = 0, zeros;
    scan2<NT>(zero, before, &zeros, &total, sh.n_sums, sh.w_sums);
    const Cuts cuts(total, most);
#pragma unroll 1
    for (int w = 0; w <= PER; ++w) {
      const long long x = cuts.at((long long)blockIdx.x * PER + w);
      if (before <= x && x < before + mine) {
        sh.own[w].b = b_t0;
        sh.own[w].t0 = t0;
        sh.own[w].before = before;
      }
    }
    __syncthreads();
    const long long x = cuts.at(worker);
    const int w = (int)(worker - (long long)blockIdx.x * PER);
    cut = {tiles, 0, 0, 0};
    b = B;
    f = tiles;
    if (x < total) {
      b = sh.own[w].b;
      have = false;
      long long from = sh.own[w].before;
#pragma unroll 1
      for (int t = sh.own[w].t0;; ++t) {
        const int cost = units_of(t);
        const long long span = (long long)(cost + g.start) * c.HKV;
        if (x < from + span) {
          cut = cut_in(g, cuts, c.HKV, t, cost, x, x - from);
          f = first[b];
          break;
        }
        from += span;
      }
    }
    __syncthreads();  // `first` is read
  }
  p.b = __shfl_sync(0xffffffffu, b, 0);
  p.first = __shfl_sync(0xffffffffu, f, 0);
  p.tile = __shfl_sync(0xffffffffu, cut.tile, 0);
  p.head = __shfl_sync(0xffffffffu, cut.head, 0);
  p.unit = __shfl_sync(0xffffffffu, cut.unit, 0);
  p.end_tile = __shfl_sync(0xffffffffu, cut.tile, 1);
  p.end_head = __shfl_sync(0xffffffffu, cut.head, 1);
  p.end_unit = __shfl_sync(0xffffffffu, cut.unit, 1);
  p.ender = __shfl_sync(0xffffffffu, cut.ender, 1);
  seq.slot = __shfl_sync(0xffffffffu, s.slot, 0);
  seq.len = __shfl_sync(0xffffffffu, s.len, 0);
  seq.row0 = __shfl_sync(0xffffffffu, s.row0, 0);
  seq.n = __shfl_sync(0xffffffffu, s.n, 0);
  return p;
}

// A worker's way along its part, an item (or what of it lies in the part) at a time.
struct Seg {
  Seq s;
  Tile x;
  int head;
  int k0, n;          // units [k0, k0 + n) of keys (n = 0: an item that sees none)
  bool starts, ends;  // the item begins / ends here
  int slot;           // of a partial result: 0 or 1
};

struct Walk {
  Part p;
  Seq s;
  bool moved;
  __device__ __forceinline__ Walk(const Part& part, const Seq& seq) : p(part), s(seq), moved(false) {}
  __device__ __forceinline__ bool done() const {
    return p.tile == p.end_tile && p.head == p.end_head && p.unit == p.end_unit;
  }
  __device__ __forceinline__ bool next(const Geo& g, const fakv_cache& c, const int* cu, const int* slots, int T, Seg& o) {
    if (done()) return false;
    if (p.unit == 0 && p.head == 0) {
      while ((p.tile - p.first) * g.R >= s.n * g.rep.d) {  // the next sequence with rows
        p.first += tiles_of(g, s.n);
        s = load_seq(c, cu, slots, ++p.b, T);
      }
    }
    o.s = s;
    o.x = tile_of(g, s, p.tile - p.first);
    o.head = p.head;
    o.slot = moved ? 1 : 0;
    const int cost = max(1, o.x.units);
    const bool cut = p.tile == p.end_tile && p.head == p.end_head;
    const int to = cut ? p.end_unit : cost;
    o.k0 = o.x.u0 + p.unit;
    o.n = min(to, o.x.units) - p.unit;
    o.starts = p.unit == 0;
    o.ends = !cut;
    moved = true;
    if (cut) {
      p.unit = to;
    } else {
      p.unit = 0;
      if (++p.head == c.HKV) { p.head = 0; ++p.tile; }
    }
    return true;
  }
};

// What worker k left of an item that it did not do whole: slot 2 k (the item its part begins
// in) or 2 k + 1 (the one it ends in); `ender` is the worker that ends the item. PART_JOINED: the CTA's workers all had one item and
// put their results together, in the first one's slot.
enum { PART_STARTS = 1, PART_ENDS = 2, PART_JOINED = 4 };
struct Left {
  int flags, row0, rho0, rows, head, ender, pad[2];
};

// Partial results: O [slots][R][D] not normalised, and per row the maximum m (log2 units)
// its exponentials were taken against and their sum l.
struct Partials {
  Left* left;
  float* O;
  float2* ml;
};

inline size_t partials_bytes(int workers, int R, int D) {
  return (size_t)workers * 2 * (sizeof(Left) + (size_t)R * (D + 2) * 4);
}
inline Partials partials_at(void* p, int workers, int R, int D) {
  Partials x;
  x.left = static_cast<Left*>(p);
  x.O = reinterpret_cast<float*>(x.left + 2 * workers);
  x.ml = reinterpret_cast<float2*>(x.O + (size_t)2 * workers * R * D);
  return x;
}

struct JoinArgs {
  Partials part;
  void* O;
  float* LSE;
  int ctas, per;   // workers: per of each CTA
  int R, D;        // rows of a slot, columns of a row
  int H, Dv, out_bf16;
  Div rep;
};
constexpr int TALL_CTAS = 256;  // CTAs that launch_join_tall takes (sm_103 parts have fewer SMs)
fa_status launch_join(const JoinArgs& a, cudaStream_t s);        // several workers to a CTA
fa_status launch_join_tall(const JoinArgs& a, cudaStream_t s);   // a CTA is a worker; many rows

}  // namespace kv
}  // namespace fa
