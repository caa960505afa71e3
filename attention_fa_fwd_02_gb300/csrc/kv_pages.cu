// kv_pages.cu -- the pages of a paged cache: growing, forking, freeing, compacting.
//
// The book-keeping is a few thousand integers and is bound by the latency of its
// dependent steps, so each list is planned by one block in one launch and the pages that
// have to move are copied by a second, launched as its programmatic dependent. Page
// copies are bound by bandwidth (2 x the bytes of the pages). Every choice depends on the
// list and on page numbers alone (prefix sums, no first-come atomics), so results are
// the same on every run.
//
// Measured: 96 samples forked from 32 sequences and grown, 24 MB of last pages copied in 4
// planes: 16.1 us (fork 4.6 by two launches, plan 7, copy 5: launches and look-ups; the copy's floor
// is 7 us); a page each for 64 slots 6.3 us in a pool of 5000 pages, 11.8 in one of 130000 and 20.3
// of 500000, all but full; 64 slots of 1024 pages freed 3.5 us, 16384 of 4 pages 59 (each entry is
// looked for in the list before it); 8192 pages closed up, 1900 of them moved in 2 planes: 92 us with
// the two small copies around it, the move itself 71 us, 490 MB at 6.9 TB/s, the rate of a copy.
#include "kv_common.cuh"

namespace fa {
namespace kv {
namespace {

constexpr int PLAN = 1024;   // threads of a planning block
constexpr int SCAN = 4;      // reference counts per thread and step
constexpr int WIDE = 16;     // and in grow's walk past the first of them
constexpr int NEAR = 4096;   // pages given to a part of a list through shared memory
constexpr int BRIEF = 256;   // entries of a list compared with one another

// Sums saturate: no list can be served more than 2^28 pages, and beyond them only "too
// many" matters.
constexpr unsigned MANY = 1u << 30;
__device__ __forceinline__ unsigned sat(unsigned x, unsigned y) { return min(x + y, MANY); }

// Exclusive prefix sum over the block (PLAN threads, values up to MANY); *total: the sum.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned* total) {
  __shared__ unsigned sums[PLAN / 32], before[PLAN / 32 + 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y = sat(y, v);
  }
  if (lane == 31) sums[w] = y;
  __syncthreads();
  if (w == 0) {
    unsigned z = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, z, d);
      if (lane >= d) z = sat(z, u);
    }
    before[lane + 1] = z;
    if (lane == 0) before[0] = 0;
  }
  __syncthreads();
  y = __shfl_up_sync(0xffffffffu, y, 1);
  const unsigned r = sat(before[w], lane ? y : 0u);
  *total = before[PLAN / 32];
  __syncthreads();
  return r;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((long long)tokens + (1 << shift) - 1) >> shift);
}

// a slot's length; -1 and the status bit where it is no length of a row: its entry is left out
__device__ __forceinline__ int length_of(const fakv_cache& c, int slot) {
  const int len = c.lens[slot];
  if (len >= 0 && (long long)len <= (long long)c.max_pages * c.page_size) return len;
  raise(c.status, FAKV_BAD_LENGTH);
  return -1;
}

// ------------------------------------------------------------------ page copies
struct CopyArgs {
  char* base[2];           // K, V
  long long plane_bytes, page_bytes;  // strides
  int planes, chunks;                 // block steps of COPY_CHUNK bytes to a page
  int bytes;                          // of a page
};

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNROLL = 4;
constexpr int COPY_CHUNK = COPY_THREADS * COPY_UNROLL * 16;

// pages pair[i].x -> pair[i].y for i < n, in every plane of K and V
__device__ __forceinline__ void copy_pages(const CopyArgs& a, const int2* pair, int n) {
  const long long per = 2ll * a.planes * a.chunks;
  for (long long w = blockIdx.x; w < n * per; w += gridDim.x) {
    const int i = (int)(w / per);
    int r = (int)(w - i * per);
    const int ch = r % a.chunks;
    r /= a.chunks;
    const int2 p = pair[i];
    char* base = a.base[r & 1] + (r >> 1) * a.plane_bytes;
    const uint4* src = reinterpret_cast<const uint4*>(base + p.x * a.page_bytes);
    uint4* dst = reinterpret_cast<uint4*>(base + p.y * a.page_bytes);
    const int end = a.bytes / 16;
    const int at = ch * (COPY_CHUNK / 16) + threadIdx.x;
    uint4 v[COPY_UNROLL];
#pragma unroll
    for (int k = 0; k < COPY_UNROLL; ++k)
      if (at + k * COPY_THREADS < end) v[k] = src[at + k * COPY_THREADS];
#pragma unroll
    for (int k = 0; k < COPY_UNROLL; ++k)
      if (at + k * COPY_THREADS < end) dst[at + k * COPY_THREADS] = v[k];
  }
}

CopyArgs copy_args(const fakv_cache& c) {
  const long long es = esize(c.dtype);
  CopyArgs a;
  a.base[0] = static_cast<char*>(c.K);
  a.base[1] = static_cast<char*>(c.V);
  a.plane_bytes = c.planes > 1 ? c.plane_stride * es : 0;  // (of one plane: any number)
  a.page_bytes = c.page_stride * es;
  a.planes = c.planes;
  a.bytes = (int)((long long)c.page_size * c.HKV * c.D * es);
  a.chunks = (a.bytes + COPY_CHUNK - 1) / COPY_CHUNK;
  return a;
}

int copy_grid(long long pages_at_most, const CopyArgs& a) {
  const long long w = pages_at_most * 2 * a.planes * a.chunks, most = 8ll * host::sm_count();
  return (int)(w < 1 ? 1 : w < most ? w : most);
}

// ------------------------------------------------------------------ grow
struct GrowArgs {
  fakv_cache c;
  const int* slots;
  const int* add;
  int n, shift;
  bool quads;  // refs may be read four at a time
  int* mark;   // scratch [max_slots]: first place of a slot in the list (lists above BRIEF)
  int* fresh;  // scratch [num_pages]: the free pages, in order (above NEAR of them)
  int2* pair;  // scratch [n]: pages to copy
  int* count;  // scratch: how many
};

// Entry i needs pages for its new tokens, and one for a shared last page with room in it.
// Prefix sums of the needs over the list give each entry its place among the free pages;
// these are ranked by walking refs upwards until the list is served. Ranks then go to
// (entry, column) by a search in the prefix, so one long entry is as parallel as many
// short ones. Released shares are taken off at the end: no page that is a copy's source
// becomes free before the copies. Lists longer than the block are taken part by part.
__global__ void __launch_bounds__(PLAN) grow_kernel(const __grid_constant__ GrowArgs a) {
  __shared__ unsigned first[PLAN];
  __shared__ int col0[PLAN], slot_of[PLAN];  // slot_of: -1 where nothing is given
  __shared__ int from_sh;
  __shared__ int near[NEAR];  // free pages of a part of the list that needs few
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  int refs0[SCAN];  // the first counts, asked for before the list is known
#pragma unroll
  for (int k = 0; k < SCAN; ++k) refs0[k] = tid * SCAN + k < a.c.num_pages ? a.c.refs[tid * SCAN + k] : 1;
  // Which entry of a slot is the first: short lists are compared in shared memory (three round
  // trips to memory less), long ones mark their slots.
  const bool brief = a.n <= BRIEF;
  if (brief) {
    if (tid < a.n) slot_of[tid] = a.slots[tid];
  } else {
    for (int i = tid; i < a.n; i += PLAN) {
      const int s = a.slots[i];
      if ((unsigned)s < (unsigned)a.c.max_slots) a.mark[s] = a.n;
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += PLAN) {
      const int s = a.slots[i];
      if ((unsigned)s < (unsigned)a.c.max_slots) atomicMin(&a.mark[s], i);
    }
  }
  __syncthreads();
  int copies = 0;         // copies listed so far
  int from = 0;           // first page not yet walked past
  bool exhausted = false; // an entry was not served: none that needs pages is, from there on
  for (int e0 = 0; e0 < a.n; e0 += PLAN) {
    const int i = e0 + tid;
    int slot = -1, len = 0, add = 0, old = 0, tail = -1;
    unsigned need = 0;
    if (i < a.n) {
      slot = brief ? slot_of[i] : a.slots[i];
      bool again = false;
      if ((unsigned)slot >= (unsigned)a.c.max_slots) {
        raise(a.c.status, FAKV_BAD_SLOT);
        slot = -1;
      } else if (brief) {
        for (int j = 0; j < i; ++j) again |= slot_of[j] == slot;
      } else {
        again = a.mark[slot] != i;
      }
      if (again) {
        raise(a.c.status, FAKV_REPEATED);
        slot = -1;
      }
    }
    if (slot >= 0) {
      len = length_of(a.c, slot);
      add = a.add[i];
      if (add < 0) raise(a.c.status, FAKV_BAD_LENGTH);
      if (len < 0 || add < 0) slot = -1;
    }
    if (slot >= 0) {
      old = pages_of(len, a.shift);
      if ((long long)len + add > (long long)a.c.max_pages * a.c.page_size) {
        raise(a.c.status, FAKV_ROW_FULL);
        slot = -1;
      } else {
        if (add > 0 && (len & (a.c.page_size - 1))) {
          const int p = page_of(a.c, slot, len, a.shift);
          if (p < 0) slot = -1;  // the new tokens would have no place
          else if (a.c.refs[p] > 1) tail = p;
        }
        if (slot >= 0) need = pages_of(len + add, a.shift) - old + (tail >= 0);
      }
    }
    unsigned total;
    const unsigned place = block_scan(need, &total);
    first[tid] = place;
    if (tid == 0) from_sh = from;
    // rank the free pages until there are `total`
    const bool few = total <= NEAR;
    unsigned got = 0;
    auto rank = [&](int page, unsigned open) {  // this thread's next pages, a bit for each free one
      unsigned here, r = got + block_scan(__popc(open), &here);
      for (; open && r < total; open &= open - 1) {
        const int free = page + __ffs(open) - 1;
        if (few) near[r] = free;
        else a.fresh[r] = free;
        if (++r == total) from_sh = free + 1;
      }
      got += here;
    };
    int at = from & ~3;
    if (e0 == 0 && total > 0) {
      unsigned open = 0;
#pragma unroll
      for (int k = 0; k < SCAN; ++k) open |= (refs0[k] == 0) << k;
      rank(tid * SCAN, open);
      at = PLAN * SCAN;
    }
    // Pools are mostly full: a step over used pages is one load of whole lines, on its way while
    // the step before it is looked at, and one barrier. Where a page is free, each thread takes
    // WIDE neighbours, so that ranks follow page numbers.
    int4 seen[WIDE / 4];
    auto four = [&](int page) {
      if (a.quads && page + 4 <= a.c.num_pages) return *reinterpret_cast<const int4*>(a.c.refs + page);
      auto one = [&](int p) { return p < a.c.num_pages ? a.c.refs[p] : 1; };
      return make_int4(one(page), one(page + 1), one(page + 2), one(page + 3));
    };
    auto ask = [&](int step) {
#pragma unroll
      for (int k = 0; k < WIDE / 4; ++k) seen[k] = four(step + (tid / 32 * WIDE + k * 4) * 32 + lane * 4);
    };
    const bool walk = !exhausted && got < total && at < a.c.num_pages;
    if (walk) ask(at);
    for (; walk && got < total && at < a.c.num_pages; at += PLAN * WIDE) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < WIDE / 4; ++k) any |= seen[k].x == 0 || seen[k].y == 0 || seen[k].z == 0 || seen[k].w == 0;
      ask(at + PLAN * WIDE);
      if (!__syncthreads_or(any)) continue;
      const int page = at + tid * WIDE;
      unsigned open = 0;
#pragma unroll
      for (int k = 0; k < WIDE; k += 4) {
        const int4 c = four(page + k);
        open |= ((c.x == 0) | (c.y == 0) << 1 | (c.z == 0) << 2 | (c.w == 0) << 3) << k;
      }
      if (page < from) open &= from - page < WIDE ? ~0u << (from - page) : 0u;
      rank(page, open);
    }
    const unsigned found = min(got, total);
    const bool served = slot >= 0 && (need == 0 || place + need <= found);
    if (slot >= 0 && !served) raise(a.c.status, FAKV_NO_PAGES);
    if (found < total) exhausted = true;
    col0[tid] = old - (tail >= 0);
    slot_of[tid] = served ? slot : -1;
    __syncthreads();
    from = from_sh;
    for (unsigned r = tid; r < found; r += PLAN) {
      int lo = 0, hi = PLAN;  // the entry of rank r: the last with first <= r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= r) lo = mid; else hi = mid;
      }
      if (slot_of[lo] < 0) continue;
      const int page = few ? near[r] : a.fresh[r];
      a.c.table[(long long)slot_of[lo] * a.c.table_stride + col0[lo] + (int)(r - first[lo])] = page;
      a.c.refs[page] = 1;
    }
    const bool copy = served && tail >= 0;
    unsigned n_copy;
    const unsigned c_at = block_scan(copy, &n_copy);
    if (copy) a.pair[copies + c_at] = make_int2(tail, few ? near[place] : a.fresh[place]);
    copies += (int)n_copy;
    if (served) a.c.lens[slot] = len + add;
    __syncthreads();
  }
  for (int i = tid; i < copies; i += PLAN) atomicSub(&a.c.refs[a.pair[i].x], 1);
  if (tid == 0) *a.count = copies;
}

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ CopyArgs a,
                                                            const int2* pair, const int* count) {
  ptx::grid_dependency_wait();
  copy_pages(a, pair, *count);
}

// ------------------------------------------------------------------ fork, free
struct ListArgs {
  fakv_cache c;
  const int* src;  // fork
  const int* dst;  // fork: destinations; free: the slots
  const int* keep; // free, may be null
  int n, shift;
  int* rows;       // fork scratch [n][max_pages]
  int* lens;       // fork scratch [n]: the sources' lengths, -1: entry left out
};

// whether entry i's slot in `list` is in range and named by no earlier entry (one block)
__device__ __forceinline__ bool entry_ok(const fakv_cache& c, const int* list, int i, int slot) {
  if ((unsigned)slot >= (unsigned)c.max_slots) {
    if (threadIdx.x == 0) raise(c.status, FAKV_BAD_SLOT);
    return false;
  }
  bool seen = false;
  for (int j = threadIdx.x; j < i; j += blockDim.x) seen |= list[j] == slot;
  if (__syncthreads_or(seen)) {
    if (threadIdx.x == 0) raise(c.status, FAKV_REPEATED);
    return false;
  }
  return true;
}

// Takes the sources' rows and counts one more holder for their pages, before anything is
// released: a page that moves from one slot of the list to another stays in use.
__global__ void __launch_bounds__(256) fork_take_kernel(const __grid_constant__ ListArgs a) {
  ptx::grid_launch_dependents();
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int src = a.src[i], dst = a.dst[i];
    bool ok = entry_ok(a.c, a.dst, i, dst);
    if (ok && (unsigned)src >= (unsigned)a.c.max_slots) {
      if (threadIdx.x == 0) raise(a.c.status, FAKV_BAD_SLOT);
      ok = false;
    }
    int len = -1;
    if (ok) {
      len = length_of(a.c, src);
      if (length_of(a.c, dst) < 0) len = -1;
    }
    if (threadIdx.x == 0) a.lens[i] = len;
    const int* row = a.c.table + (long long)src * a.c.table_stride;
    for (int k = threadIdx.x; len > 0 && k < pages_of(len, a.shift); k += blockDim.x) {
      const int p = row[k];
      a.rows[(long long)i * a.c.max_pages + k] = p;
      if ((unsigned)p < (unsigned)a.c.num_pages) atomicAdd(&a.c.refs[p], 1);
      else raise(a.c.status, FAKV_BAD_PAGE);
    }
  }
}

// columns [from, to) of a slot's row released
__device__ __forceinline__ void release(const fakv_cache& c, int* row, int from, int to) {
  for (int k = from + threadIdx.x; k < to; k += blockDim.x) {
    const int p = row[k];
    if ((unsigned)p < (unsigned)c.num_pages) atomicSub(&c.refs[p], 1);
    else raise(c.status, FAKV_BAD_PAGE);
    row[k] = -1;
  }
}

__global__ void __launch_bounds__(256) fork_give_kernel(const __grid_constant__ ListArgs a) {
  ptx::grid_dependency_wait();
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int len = a.lens[i];
    if (len < 0) continue;
    const int dst = a.dst[i];
    int* row = a.c.table + (long long)dst * a.c.table_stride;
    release(a.c, row, 0, pages_of(a.c.lens[dst], a.shift));
    __syncthreads();
    for (int k = threadIdx.x; k < pages_of(len, a.shift); k += blockDim.x)
      row[k] = a.rows[(long long)i * a.c.max_pages + k];
    if (threadIdx.x == 0) a.c.lens[dst] = len;
  }
}

// Short lists of short rows in one launch of one block: a warp per entry, rows in registers.
// Three dependent look-ups and no scratch: 3 entries of 21 pages 2.3 us, 32 of 250 4.4 (two
// launches, whose time hardly depends on either: 4.0 and 4.7).
constexpr int SHORT_LIST = PLAN / 32;  // entries
constexpr int SHORT_STEPS = 8;         // 32 pages each
__global__ void __launch_bounds__(PLAN) fork_short_kernel(const __grid_constant__ ListArgs a) {
  const int i = threadIdx.x / 32, lane = threadIdx.x & 31;
  int dst = -1, len = -1, now = 0, was = 0;
  int take[SHORT_STEPS], held[SHORT_STEPS];
  if (i < a.n) {
    const int other = lane < a.n ? a.dst[lane] : -1;
    const int src = a.src[i];
    dst = __shfl_sync(0xffffffffu, other, i);
    const bool in = (unsigned)dst < (unsigned)a.c.max_slots;
    const bool again = __any_sync(0xffffffffu, lane < i && other == dst);
    const bool ok = in && !again && (unsigned)src < (unsigned)a.c.max_slots;
    if (!ok && lane == 0) raise(a.c.status, in && again ? FAKV_REPEATED : FAKV_BAD_SLOT);
    if (ok) {
      len = length_of(a.c, src);
      const int held_len = length_of(a.c, dst);
      if (held_len < 0) len = -1;
      now = len < 0 ? 0 : pages_of(len, a.shift);
      was = len < 0 ? 0 : pages_of(held_len, a.shift);
      const int* from = a.c.table + (long long)src * a.c.table_stride;
      const int* to = a.c.table + (long long)dst * a.c.table_stride;
#pragma unroll
      for (int s = 0; s < SHORT_STEPS; ++s) {
        const int k = 32 * s + lane;
        take[s] = k < now ? from[k] : -1;
        held[s] = k < was ? to[k] : -1;
      }
#pragma unroll
      for (int s = 0; s < SHORT_STEPS; ++s) {
        const int k = 32 * s + lane;
        if (k < now) {
          if ((unsigned)take[s] < (unsigned)a.c.num_pages) atomicAdd(&a.c.refs[take[s]], 1);
          else raise(a.c.status, FAKV_BAD_PAGE);
        }
        if (k < was) {
          if ((unsigned)held[s] < (unsigned)a.c.num_pages) atomicSub(&a.c.refs[held[s]], 1);
          else raise(a.c.status, FAKV_BAD_PAGE);
        }
      }
    }
  }
  __syncthreads();  // every row and length is read
  if (len < 0) return;
  int* row = a.c.table + (long long)dst * a.c.table_stride;
#pragma unroll
  for (int s = 0; s < SHORT_STEPS; ++s) {
    const int k = 32 * s + lane;
    if (k < max(now, was)) row[k] = take[s];
  }
  if (lane == 0) a.c.lens[dst] = len;
}

__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ ListArgs a) {
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int slot = a.dst[i];
    if (!entry_ok(a.c, a.dst, i, slot)) continue;
    const int len = length_of(a.c, slot);
    if (len < 0) continue;
    int keep = a.keep ? a.keep[i] : 0;
    if (keep < 0) {
      if (threadIdx.x == 0) raise(a.c.status, FAKV_BAD_LENGTH);
      continue;
    }
    keep = min(keep, len);
    __syncthreads();  // every thread has read the length
    release(a.c, a.c.table + (long long)slot * a.c.table_stride, pages_of(keep, a.shift),
            pages_of(len, a.shift));
    if (threadIdx.x == 0) a.c.lens[slot] = keep;
  }
}

// ------------------------------------------------------------------ compact
struct CompactArgs {
  fakv_cache c;
  CopyArgs copy;
  int* to;     // scratch [num_pages]: where a page went
  int2* pair;  // scratch [num_pages]
  int* count;  // scratch: how many moves
};

__global__ void __launch_bounds__(PLAN) compact_plan_kernel(const __grid_constant__ CompactArgs a) {
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, N = a.c.num_pages;
  int movers = 0;
  const int per = (N + PLAN - 1) / PLAN;
  if (per <= 64) {
    // a run of pages per thread, read once: which of them are used, as bits
    const int p0 = min(N, tid * per), n = min(N, p0 + per) - p0;
    unsigned long long used = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) used |= (unsigned long long)(a.c.refs[p0 + k] > 0) << k;
    unsigned L_;
    block_scan((unsigned)__popcll(used), &L_);
    const int low = max(0, min((int)L_ - p0, n));  // pages of the run below L
    const unsigned long long below = low == 64 ? ~0ull : (1ull << low) - 1;
    unsigned long long hole = ~used & below, mover = used & ~below;
    unsigned moves;
    for (int i = (int)block_scan((unsigned)__popcll(hole), &moves); hole; hole &= hole - 1)
      a.pair[i++].y = p0 + __ffsll((long long)hole) - 1;
    for (int i = (int)block_scan((unsigned)__popcll(mover), &moves); mover; mover &= mover - 1)
      a.pair[i++].x = p0 + __ffsll((long long)mover) - 1;
    for (int k = 0; k < n; ++k) a.to[p0 + k] = p0 + k;
    movers = (int)moves;
  } else {
    unsigned live = 0;
    for (int at = tid; at < N; at += PLAN) live += a.c.refs[at] > 0;
    unsigned L_;
    block_scan(live, &L_);
    const int L = (int)L_;
    int holes = 0;  // ranked so far (as many as movers in the end)
    for (int at = 0; at < N; at += PLAN * SCAN) {
      int h = 0, m = 0;
      bool used[SCAN];
#pragma unroll
      for (int k = 0; k < SCAN; ++k) {
        const int p = at + tid * SCAN + k;
        used[k] = p < N && a.c.refs[p] > 0;
        if (p < N) { h += p < L && !used[k]; m += p >= L && used[k]; }
      }
      // at most PLAN * SCAN of each in a step: both fit one word
      unsigned both;
      const unsigned r = block_scan((unsigned)(h | (m << 16)), &both);
      int rh = holes + (int)(r & 0xffff), rm = movers + (int)(r >> 16);
#pragma unroll
      for (int k = 0; k < SCAN; ++k) {
        const int p = at + tid * SCAN + k;
        if (p >= N) break;
        if (p < L && !used[k]) a.pair[rh++].y = p;
        if (p >= L && used[k]) a.pair[rm++].x = p;
        a.to[p] = p;
      }
      holes += (int)(both & 0xffff);
      movers += (int)(both >> 16);
    }
  }
  __syncthreads();
  for (int i = tid; i < movers; i += PLAN) {
    const int2 p = a.pair[i];
    a.to[p.x] = p.y;
    a.c.refs[p.y] = a.c.refs[p.x];
    a.c.refs[p.x] = 0;
  }
  if (tid == 0) a.count[0] = movers;
}

// The rows renumbered and the pages moved (sources lie above every destination). Whole rows, a
// step of STEP entries at a time: an entry past its row's length goes on naming its page too.
__global__ void __launch_bounds__(COPY_THREADS) compact_move_kernel(const __grid_constant__ CompactArgs a) {
  ptx::grid_dependency_wait();
  constexpr int STEP = 1024;
  const long long steps = (a.c.max_pages + STEP - 1) / STEP;
  for (long long w = blockIdx.x; w < a.c.max_slots * steps; w += gridDim.x) {
    const long long s = w / steps;
    const int from = (int)(w - s * steps) * STEP;
    int* row = a.c.table + s * a.c.table_stride;
    for (int k = from + threadIdx.x; k < min(a.c.max_pages, from + STEP); k += blockDim.x) {
      const int p = row[k];
      if ((unsigned)p < (unsigned)a.c.num_pages) {
        const int q = a.to[p];
        if (q != p) row[k] = q;
      }
    }
  }
  copy_pages(a.copy, a.pair, a.count[0]);
}

// Stream-ordered scratch that is given back when it goes out of scope.
struct Scratch {
  char* p = nullptr;
  cudaStream_t s;
  bool ok;
  Scratch(size_t bytes, cudaStream_t s_) : s(s_) {
    void* q = nullptr;
    ok = host::scratch_alloc(&q, bytes, s) == cudaSuccess;
    p = static_cast<char*>(q);
  }
  ~Scratch() { if (ok) host::scratch_free(p, s); }
};

}  // namespace

fa_status launch_grow(const fakv_cache& c, const int* slots, const int* add, int n, cudaStream_t s) {
  const size_t pair = 16, fresh = pair + (size_t)n * 8, mark = fresh + (size_t)c.num_pages * 4;
  Scratch w(mark + (size_t)c.max_slots * 4, s);
  if (!w.ok) return failed();
  GrowArgs a = {c, slots, add, n, log2_of(c.page_size), reinterpret_cast<uintptr_t>(c.refs) % 16 == 0,
                reinterpret_cast<int*>(w.p + mark),
                reinterpret_cast<int*>(w.p + fresh), reinterpret_cast<int2*>(w.p + pair),
                reinterpret_cast<int*>(w.p)};
  fa_status st;
  {
    host::KernelTimer t("grow", s);
    st = launch(grow_kernel, 1, PLAN, 0, s, a);
  }
  if (st != FA_OK) return st;  // (no plan: its scratch says nothing)
  const CopyArgs ca = copy_args(c);
  host::KernelTimer t("grow_copy", s);
  return launch_dependent(copy_kernel, copy_grid(n, ca), COPY_THREADS, s, ca, a.pair, a.count);
}

fa_status launch_fork(const fakv_cache& c, const int* src, const int* dst, int n, cudaStream_t s) {
  if (n <= SHORT_LIST && c.max_pages <= 32 * SHORT_STEPS) {
    const ListArgs b = {c, src, dst, nullptr, n, log2_of(c.page_size), nullptr, nullptr};
    host::KernelTimer t("fork_short", s);
    return launch(fork_short_kernel, 1, PLAN, 0, s, b);
  }
  const size_t rows = (size_t)n * c.max_pages * 4;
  Scratch w(rows + (size_t)n * 4, s);
  if (!w.ok) return failed();
  ListArgs a = {c, src, dst, nullptr, n, log2_of(c.page_size), reinterpret_cast<int*>(w.p),
                reinterpret_cast<int*>(w.p + rows)};
  const int grid = n < 8 * host::sm_count() ? n : 8 * host::sm_count();
  fa_status st;
  {
    host::KernelTimer t("fork_take", s);
    st = launch(fork_take_kernel, grid, 256, 0, s, a);
  }
  if (st != FA_OK) return st;
  host::KernelTimer t("fork_give", s);
  return launch_dependent(fork_give_kernel, grid, 256, s, a);
}

fa_status launch_free(const fakv_cache& c, const int* slots, const int* keep, int n, cudaStream_t s) {
  ListArgs a = {c, nullptr, slots, keep, n, log2_of(c.page_size), nullptr, nullptr};
  const int grid = n < 8 * host::sm_count() ? n : 8 * host::sm_count();
  host::KernelTimer t("free", s);
  return launch(free_kernel, grid, 256, 0, s, a);
}

fa_status launch_compact(const fakv_cache& c, cudaStream_t s) {
  Scratch w((size_t)c.num_pages * 12 + 16, s);
  if (!w.ok) return failed();
  CompactArgs a = {c, copy_args(c), reinterpret_cast<int*>(w.p + (size_t)c.num_pages * 8),
                   reinterpret_cast<int2*>(w.p), reinterpret_cast<int*>(w.p + (size_t)c.num_pages * 12)};
  fa_status st;
  {
    host::KernelTimer t("compact_plan", s);
    st = launch(compact_plan_kernel, 1, PLAN, 0, s, a);
  }
  if (st != FA_OK) return st;
  host::KernelTimer t("compact_move", s);
  return launch_dependent(compact_move_kernel, copy_grid(c.num_pages, a.copy), COPY_THREADS, s, a);
}

}  // namespace kv
}  // namespace fa
