// kv_common.cuh -- what the paged-cache kernels share: finding a row's sequence, table
// look-ups with their checks, launch declarations.
#pragma once
#include <atomic>
#include <cstdint>
#include "fa_common.cuh"
#include "fakv.h"
#include "ptx.cuh"

namespace fa {
namespace host {
// A 4-D tensor map of 16-bit elements (innermost dimension without gaps, the others'
// strides in bytes), 128-byte swizzle or none, zeros outside.
bool encode_tiled_4d(CUtensorMap* map, const void* base, const uint64_t (&dims)[4],
                     const uint64_t (&strides)[3], const uint32_t (&box)[4], bool swizzle = true);
}  // namespace host

namespace kv {

__device__ __forceinline__ void raise(int* status, int bit) {
  if (status) atomicOr(status, bit);
}

// A sequence of a call as the kernels see it. A slot out of range, or a length outside
// the row, leaves an empty one.
struct Seq {
  int slot;   // -1: none
  int len;    // tokens, the new ones included
  int row0;   // first row of q
  int n;      // new tokens; -1: cu decreases here (then sequences may overlap: no work is
              // planned from such a cu, as its tiles could number more than an int holds)
};

__device__ __forceinline__ Seq load_seq(const fakv_cache& c, const int* cu, const int* slots, int b,
                                        int T) {
  const int r0 = cu[b], r1 = cu[b + 1];
  const int slot = slots ? slots[b] : b;
  const bool ok = slot >= 0 && slot < c.max_slots;
  const int len = c.lens[ok ? slot : 0];  // (asked for before anything waits)
  const bool len_ok = len >= 0 && (long long)len <= (long long)c.max_pages * c.page_size;
  Seq s;
  s.row0 = max(0, min(r0, T));
  s.n = r1 < r0 ? -1 : max(0, min(r1, T) - s.row0);
  s.slot = ok ? slot : -1;
  s.len = ok && len_ok ? len : 0;
  if (s.n < 0) raise(c.status, FAKV_BAD_LENGTH);
  if (s.n > 0 && !(ok && len_ok)) raise(c.status, ok ? FAKV_BAD_LENGTH : FAKV_BAD_SLOT);
  return s;
}

// page of token position `pos` of slot `slot` (both in range), or -1 with the status bit
__device__ __forceinline__ int page_of(const fakv_cache& c, int slot, int pos, int shift) {
  const int p = c.table[(long long)slot * c.table_stride + (pos >> shift)];
  if ((unsigned)p < (unsigned)c.num_pages) return p;
  raise(c.status, FAKV_BAD_PAGE);
  return -1;
}

// cos and sin of pos * freq turns (see the head of kv_rope.cu)
__device__ __forceinline__ float2 turn(long long pos, unsigned long long freq) {
  const unsigned long long t = (unsigned long long)pos * freq;
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);
  const long long rest = (long long)(t - ((unsigned long long)quarter << 62));
  float s, c;
  sincospif((float)(int)(rest >> 30) * 0x1p-33f, &s, &c);  // the angle in units of pi
  if (quarter & 1) { const float x = c; c = -s; s = x; }
  if (quarter & 2) { c = -c; s = -s; }
  return make_float2(c, s);
}

// The sequence of row t: the last b with cu[b] <= t (32 probes per round, one warp), or
// -1 for rows past the last sequence. cu is probed inside [0, B] whatever it holds.
__device__ __forceinline__ int find_seq(const int* cu, int B, int t) {
  const int lane = ptx::lane_id();
  if (t >= cu[B]) return -1;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < n && cu[at] <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, below));
    if (hits == 0) return -1;
    const int first = (hits - 1) * step;
    n = min(step, n - first);
    lo += first;
  }
  return cu[lo] <= t ? lo : -1;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Dynamic shared memory of `kernel` raised to `bytes`, once per kernel and device (`done`: a
// word of the kernel's own).
template <typename K>
inline bool allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// An allocation or a launch failed: the runtime's record of it is cleared, so that the next
// call's check of its launches does not find it.
inline fa_status failed() {
  (void)cudaGetLastError();
  return FA_ERR_CUDA;
}

// The launch's own answer, not the runtime's record of the last error, which may be another call's.
template <typename... KArgs, typename... Args>
inline fa_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? FA_OK : failed();
}
// As the programmatic dependent of the launch before it (fa_common.cuh).
template <typename... KArgs, typename... Args>
inline fa_status launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  return launch_programmatic(kernel, grid, block, stream, args...) == cudaSuccess ? FA_OK : failed();
}

inline int esize(fa_dtype t) { return t == FA_BF16 ? 2 : 4; }

// launchers (arguments validated in kv_api.cu)
fa_status launch_rope(const void* q, const void* k, void* qo, void* ko, const void* pos,
                      const fakv_rope& r, const fakv_rope_params& p, cudaStream_t s);
fa_status launch_append(const void* q, const void* k, const void* v, void* qo, const int* cu,
                        const int* slots, const fakv_rope* r, const fakv_cache& c,
                        const fakv_tokens& p, cudaStream_t s);
fa_status launch_attend_rows(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                             const fakv_cache& c, const fakv_tokens& p, cudaStream_t s);
fa_status launch_attend_tiles(const void* q, void* O, float* LSE, const int* cu, const int* slots,
                              const fakv_cache& c, const fakv_tokens& p, cudaStream_t s);
fa_status launch_grow(const fakv_cache& c, const int* slots, const int* add, int n, cudaStream_t s);
fa_status launch_fork(const fakv_cache& c, const int* src, const int* dst, int n, cudaStream_t s);
fa_status launch_free(const fakv_cache& c, const int* slots, const int* keep, int n, cudaStream_t s);
fa_status launch_compact(const fakv_cache& c, cudaStream_t s);
unsigned int read_and_clear_kv_status(cudaError_t* err);
unsigned int read_and_clear_kvq_status(cudaError_t* err);

}  // namespace kv
}  // namespace fa
