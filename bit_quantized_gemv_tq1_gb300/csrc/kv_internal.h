// kv_internal.h -- host-side launchers of the paged key/value cache's
// operators (rotary append, attention, page bookkeeping) and the structures
// they hand to their kernels.  Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq1 {

enum : int { kF32 = 0, kF16 = 1, kBf16 = 2 };  // element types, as enum tq1_dtype

// Device status bits beside kStatusTimeout and kStatusBadId.
enum : unsigned { kStatusNoPages = 4u };

// Address of the library's device status word on the current device, or
// nullptr when a runtime call failed.
unsigned* status_word();

// A divisor of non-negative 32-bit integers that the host knows, with its
// reciprocal (Granlund and Montgomery, 1994): n / d = (hi(n mul) + n) >> shift
// with 2^shift >= d > 2^(shift - 1) and mul = floor(2^32 (2^shift - d) / d) + 1.
// What a kernel computes before its first loads or between those that follow
// one another is as long as its instructions, and the compiler's divisions were
// the larger part of them.
struct Divisor {
  int d, shift;
  uint32_t mul;
  Divisor() = default;
  explicit Divisor(int v) : d(v), shift(0) {
    while ((int64_t{1} << shift) < v) ++shift;
    mul = static_cast<uint32_t>((((uint64_t{1} << shift) - static_cast<uint64_t>(v)) << 32) / static_cast<uint64_t>(v)) + 1;
  }
  __host__ __device__ __forceinline__ operator int() const { return d; }
};
#ifdef __CUDACC__
__device__ __forceinline__ int operator/(int n, const Divisor& v) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), v.mul) + static_cast<uint32_t>(n)) >> v.shift);
}
#endif

struct KvCache {
  uint16_t *k, *v;                                 // 16-bit elements
  int64_t page_stride, head_stride, slot_stride;   // elements
  int n_pages, n_kv, page_size, page_shift, d, dtype;
};

struct KvBatch {
  const int32_t *table, *q_start, *kv_len;
  int n_seqs, max_pages;
  int t;        // rows of the call's tensors
  int max_len;  // slots a table row addresses
};

struct RopeArgs {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;  // elements between tokens
  uint16_t* q_out;        // [t][n_q][d]
  const float* inv_freq;
  const int32_t* positions;
  int n_q, rot, interleaved, in_dtype;
  float mscale;
};

int launch_rope_freqs(float* inv_freq, int rot, double base, double factor, double orig_len, double low, double high,
                      cudaStream_t s);
int launch_rope_append(const KvCache& c, const KvBatch& b, const RopeArgs& a, unsigned* status, cudaStream_t s);

struct AttnArgs {
  const uint16_t* q;
  void* out;
  int64_t ldq, ldo;  // elements between tokens
  float scale;
  int n_q, causal, window, out_f32;
};

struct Part;  // kv.cuh

// The 128-row tensor-core kernel (`pair`: two such tiles side by side).
// Returns TQ1_ERR_UNSUPPORTED, launching nothing, for strides that a tensor
// map cannot describe.
int launch_attn_tile(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool pair, int ctas, Part* parts,
                     float* slots, unsigned* status, cudaStream_t s);
int attn_tile_rows(int group, bool pair);

size_t attn_workspace_bytes(const KvCache& c, int64_t t, int64_t n_q, int64_t n_seqs);
int launch_attn(const KvCache& c, const KvBatch& b, const AttnArgs& a, void* ws, unsigned* status, cudaStream_t s);

struct PagePool {
  uint8_t* base;
  int64_t pool_stride, page_bytes;
  int32_t *table, *kv_len, *refs;
  int n_pools, n_pages, n_seqs, max_pages;
  Divisor page_size;
};

size_t pages_workspace_bytes(int64_t n_pages, int64_t n_seqs);
int launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int64_t n, unsigned* status,
                      cudaStream_t s);
int launch_pages_resize(const PagePool& p, const int32_t* seqs, const int32_t* lens, int n, void* ws, unsigned* status,
                        cudaStream_t s);
int launch_pages_fork(const PagePool& p, const int32_t* parents, const int32_t* children, int n, void* ws,
                      unsigned* status, cudaStream_t s);
int launch_pages_compact(const PagePool& p, void* ws, unsigned* status, cudaStream_t s);

}  // namespace tq1
