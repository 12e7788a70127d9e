// pages.cu -- page bookkeeping of the key/value cache: growing, shrinking and
// freeing sequences, forking them with shared pages, compacting the pool, and
// the page copies these ask for.
//
// State (device memory, the caller's): a table row of page ids and a length
// per sequence, and refs[p] = how many sequences hold page p.  A page is free
// exactly when refs[p] == 0, so there is no list to keep in step: allocation
// takes the lowest free ids, in the order of the call's arguments, and every
// result is determined by the arguments.
//
// A bookkeeping kernel changes the tables and writes the list of page copies
// (source, destination) to the workspace; the copy kernel that follows moves
// each page of the list in every pool (keys and values of all layers share
// one set of tables).  A list never names a page both as source and as
// destination: destinations were free, sources were not.
//
// Bound: the copies by HBM (each byte read and written once); the
// bookkeeping, a few thousand integers, by latency, which is why resize and
// fork do theirs in one CTA.
#include "../../include/tq1.h"
#include "kv.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kChunkPages = 4 * kPlanThreads;  // pages of one compaction chunk
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                    // 16-byte pieces per thread and step
constexpr int kCopyBytes = kCopyThreads * kCopyVecs * 16;       // bytes of one step of a CTA

// Workspace: a header of 64 words, the copy list, and per-page / per-argument
// scratch.
struct PagesWs {
  int32_t* count;   // [0]: copies in the list; compaction: [1] live pages, [2] pages to move
  int32_t* src;     // [n_pages]
  int32_t* dst;     // [n_pages]
  int32_t* rank;    // [n_pages]   compaction: place of a moving page in the list
  int32_t* chunks;  // [ceil(n_pages / kChunkPages)] live pages per chunk
  int32_t* need;    // [n_seqs]    pages wanted before argument i; [n_seqs] flags follow
};
__host__ __device__ inline size_t pages_words(int64_t n_pages, int64_t n_seqs) {
  return 64 + 3 * static_cast<size_t>(n_pages) + (n_pages + kChunkPages - 1) / kChunkPages + 2 * static_cast<size_t>(n_seqs);
}
inline PagesWs split_ws(void* ws, int64_t n_pages) {
  PagesWs w;
  w.count = static_cast<int32_t*>(ws);
  w.src = w.count + 64;
  w.dst = w.src + n_pages;
  w.rank = w.dst + n_pages;
  w.chunks = w.rank + n_pages;
  w.need = w.chunks + (n_pages + kChunkPages - 1) / kChunkPages;
  return w;
}

__device__ __forceinline__ int up(int a, int b) { return (a + b - 1) / b; }

// The lowest `want` free pages into `out`, ascending, by the whole CTA; the
// scan stops as soon as it has them.  Returns how many there were (<= want).
__device__ int find_free(const int32_t* refs, int n_pages, int want, int32_t* out, int* s_warp) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += kChunkPages) {
    const int p0 = base + 4 * threadIdx.x;
    int r[4] = {1, 1, 1, 1};
    if (p0 + 3 < n_pages) {
      const int4 v = __ldcg(reinterpret_cast<const int4*>(refs + p0));
      r[0] = v.x;
      r[1] = v.y;
      r[2] = v.z;
      r[3] = v.w;
    } else {
      for (int i = 0; i < 4; ++i)
        if (p0 + i < n_pages) r[i] = __ldcg(refs + p0 + i);
    }
    const int mine = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int total;
    int at = found + block_scan<kPlanThreads>(mine, s_warp, total) - mine;
    for (int i = 0; i < 4; ++i)
      if (r[i] == 0) {
        if (at < want) out[at] = p0 + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// Exclusive sums of need[i] (n values, in place), by the whole CTA; returns
// their total, at most 2^30.
__device__ int sum_needs(int32_t* need, int n, int* s_warp) {
  int64_t before = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int v = i < n ? need[i] : 0;
    int total;
    const int end = block_scan<kPlanThreads>(v, s_warp, total);
    if (i < n) need[i] = static_cast<int32_t>(min(before + end - v, static_cast<int64_t>(1) << 30));
    before += total;
  }
  __syncthreads();
  return static_cast<int>(min(before, static_cast<int64_t>(1) << 30));
}

// Set the length of sequences seqs[i] to lens[i].
//   1. pages past a shorter length are let go;
//   2. each growing sequence's need: the pages it lacks, and one more where
//      its last page is partly filled and shared (it will write into it);
//   3. the lowest free pages are dealt to the sequences in order; from the
//      first one on that they do not suffice for, none grows (TQ1_ERR_NO_PAGES);
//   4. tables, counts, lengths; shared last pages are listed for copying.
__global__ void __launch_bounds__(kPlanThreads) resize_kernel(const PagePool p, const int32_t* seqs, const int32_t* lens,
                                                              int n, PagesWs w, unsigned* status) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_copies;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* before = w.need;
  int32_t* flag = w.need + n;  // 0: nothing to do, 1: grows, 2: grows out of a shared page
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) s_copies = 0;
  // 1: a warp per sequence, a lane per page.
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    const int s = seqs[i];
    if (s < 0 || s >= p.n_seqs) {
      if (lane == 0) raise_status(status, kStatusBadId);
      continue;
    }
    const int len = p.kv_len[s], want = lens[i];
    if (want < 0 || up(want, p.page_size) > p.max_pages || want > len) continue;
    const int had = min(up(max(len, 0), p.page_size), p.max_pages), keep = up(want, p.page_size);
    int32_t* row = p.table + static_cast<int64_t>(s) * p.max_pages;
    for (int j = keep + lane; j < had; j += 32) {
      const int id = row[j];
      if (id >= 0 && id < p.n_pages)
        atomicSub(p.refs + id, 1);
      else
        raise_status(status, kStatusBadId);
      row[j] = -1;
    }
    if (lane == 0) p.kv_len[s] = want;
  }
  __syncthreads();
  // 2
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = seqs[i];
    int need = 0, f = 0;
    if (s >= 0 && s < p.n_seqs) {
      const int len = max(p.kv_len[s], 0), want = lens[i];
      if (want < 0 || up(want, p.page_size) > p.max_pages) {
        raise_status(status, kStatusNoPages);
      } else if (want > len) {
        const int had = up(len, p.page_size);
        f = 1;
        need = up(want, p.page_size) - had;
        if (len % p.page_size != 0) {
          const int id = p.table[static_cast<int64_t>(s) * p.max_pages + had - 1];
          if (id >= 0 && id < p.n_pages && __ldcg(p.refs + id) > 1) {
            f = 2;
            ++need;
          }
        }
      }
    }
    before[i] = need;
    flag[i] = f;
  }
  __syncthreads();
  const int total = sum_needs(before, n, s_warp);
  const int have = total ? find_free(p.refs, p.n_pages, min(total, p.n_pages), w.rank, s_warp) : 0;
  // 4
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    if (flag[i] == 0) continue;
    const int s = seqs[i], len = max(p.kv_len[s], 0), want = lens[i];
    const int had = up(len, p.page_size), shared = flag[i] == 2;
    const int first = had - shared, upto = up(want, p.page_size), at = before[i];
    if (at + (upto - first) > have) {
      if (lane == 0) raise_status(status, kStatusNoPages);
      continue;
    }
    int32_t* row = p.table + static_cast<int64_t>(s) * p.max_pages;
    for (int j = first + lane; j < upto; j += 32) {
      const int id = w.rank[at + j - first];
      if (shared && j == first) {
        const int k = atomicAdd(&s_copies, 1), old = row[j];
        w.src[k] = old;
        w.dst[k] = id;
        atomicSub(p.refs + old, 1);
      }
      row[j] = id;
      p.refs[id] = 1;
    }
    if (lane == 0) p.kv_len[s] = want;
  }
  __syncthreads();
  if (threadIdx.x == 0) w.count[0] = s_copies;
}

// children[i] becomes a copy of parents[i]: whole pages shared, a partly
// filled last page copied to the lowest free one.
__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const PagePool p, const int32_t* parents,
                                                            const int32_t* children, int n, PagesWs w, unsigned* status) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_copies;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* before = w.need;
  int32_t* flag = w.need + n;  // 1: a fork
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) s_copies = 0;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = parents[i], c = children[i];
    int need = 0, f = 0;
    if (s < 0 || s >= p.n_seqs || c < 0 || c >= p.n_seqs || p.kv_len[c] != 0) {
      raise_status(status, kStatusBadId);
    } else {
      const int len = p.kv_len[s];
      f = len > 0 && up(len, p.page_size) <= p.max_pages;
      need = f && len % p.page_size != 0;
    }
    before[i] = need;
    flag[i] = f;
  }
  __syncthreads();
  const int total = sum_needs(before, n, s_warp);
  const int have = total ? find_free(p.refs, p.n_pages, min(total, p.n_pages), w.rank, s_warp) : 0;
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    if (flag[i] == 0) continue;
    const int s = parents[i], c = children[i], len = p.kv_len[s];
    const int full = len / p.page_size, part = len % p.page_size != 0, at = before[i];
    if (at + part > have) {
      if (lane == 0) raise_status(status, kStatusNoPages);
      continue;
    }
    const int32_t* from = p.table + static_cast<int64_t>(s) * p.max_pages;
    int32_t* to = p.table + static_cast<int64_t>(c) * p.max_pages;
    for (int j = lane; j < full; j += 32) {
      const int id = from[j];
      to[j] = id;
      if (id >= 0 && id < p.n_pages)
        atomicAdd(p.refs + id, 1);
      else
        raise_status(status, kStatusBadId);
    }
    if (lane == 0) {
      if (part) {
        const int id = w.rank[at], old = from[full];
        if (old >= 0 && old < p.n_pages) {
          const int k = atomicAdd(&s_copies, 1);
          w.src[k] = old;
          w.dst[k] = id;
        } else {
          raise_status(status, kStatusBadId);
        }
        to[full] = id;
        p.refs[id] = 1;
      }
      p.kv_len[c] = len;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) w.count[0] = s_copies;
}

// ------------------------------------------------------------ compaction --
// With L live pages, the j-th live page at or past L moves to the j-th free
// page below L.  First the live pages of each chunk are counted; then every
// chunk finds, from the counts of all, the place of each of its holes and
// movers; then pages, tables and counts follow.
__device__ __forceinline__ int load_live4(const int32_t* refs, int n_pages, int p0, int (&r)[4]) {
  int live = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = p0 + i < n_pages ? __ldcg(refs + p0 + i) : 0;
    live += r[i] > 0;
  }
  return live;
}

__global__ void __launch_bounds__(kPlanThreads) compact_count_kernel(const PagePool p, PagesWs w) {
  __shared__ int s_warp[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  int r[4], total;
  const int live = load_live4(p.refs, p.n_pages, blockIdx.x * kChunkPages + 4 * threadIdx.x, r);
  (void)block_scan<kPlanThreads>(live, s_warp, total);
  if (threadIdx.x == 0) w.chunks[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagePool p, PagesWs w) {
  __shared__ int s_warp[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  // Live pages in all, and in the chunks before this one and before L's.
  const int chunks = gridDim.x, me = blockIdx.x;
  const int v = threadIdx.x < chunks ? __ldcg(w.chunks + threadIdx.x) : 0;
  int L, before_me, below, r[4], t;
  (void)block_scan<kPlanThreads>(v, s_warp, L);
  (void)block_scan<kPlanThreads>(static_cast<int>(threadIdx.x) < me ? v : 0, s_warp, before_me);
  const int cl = L / kChunkPages;
  (void)block_scan<kPlanThreads>(static_cast<int>(threadIdx.x) < cl ? v : 0, s_warp, below);
  if (L % kChunkPages != 0) {
    const int p0 = cl * kChunkPages + 4 * threadIdx.x;
    (void)load_live4(p.refs, p.n_pages, p0, r);
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += p0 + i < L && r[i] > 0;
    (void)block_scan<kPlanThreads>(n, s_warp, t);
    below += t;
  }
  const int p0 = me * kChunkPages + 4 * threadIdx.x;
  const int live = load_live4(p.refs, p.n_pages, p0, r);
  int rank = before_me + block_scan<kPlanThreads>(live, s_warp, t) - live;  // live pages before p0
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = p0 + i;
    if (id >= p.n_pages) break;
    if (id < L) {
      if (r[i] <= 0) w.dst[id - rank] = id;
    } else {
      if (r[i] > 0) w.src[rank - below] = id;
      w.rank[id] = r[i] > 0 ? rank - below : -1;
    }
    rank += r[i] > 0;
  }
  if (me == 0 && threadIdx.x == 0) {
    w.count[0] = L - below;
    w.count[1] = L;
  }
}

// ---------------------------------------------------------------- copies --
// Every page of the list in every pool, in steps of kCopyBytes dealt to the
// CTAs in order; and, after a compaction plan, the tables' and counts'
// renaming, which touches nothing that is copied.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagePool p, const int32_t* count, int64_t n_fixed,
                                                                  const int32_t* src, const int32_t* dst,
                                                                  const int32_t* rank, unsigned* status) {
  pdl_wait();
  const int64_t n = count ? __ldcg(count) : n_fixed;
  if (n == 0) return;
  if (rank) {
    const int live = __ldcg(count + 1);
    const int64_t entries = static_cast<int64_t>(p.n_seqs) * p.max_pages, stride = static_cast<int64_t>(gridDim.x) * kCopyThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
    for (int64_t i = first; i < entries; i += stride) {
      const int id = p.table[i];
      if (id < live || id >= p.n_pages) continue;
      const int j = __ldcg(rank + id);
      if (j >= 0) p.table[i] = __ldcg(dst + j);
    }
    for (int64_t j = first; j < n; j += stride) {
      const int from = __ldcg(src + j);
      p.refs[__ldcg(dst + j)] = p.refs[from];
      p.refs[from] = 0;
    }
  }
  const int steps = static_cast<int>((p.page_bytes + kCopyBytes - 1) / kCopyBytes);  // of one page
  const int64_t all = n * p.n_pools * steps;
  for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
    const int64_t pg = u / steps;
    const int step = static_cast<int>(u - pg * steps);
    const int64_t i = pg % n, pool = pg / n;
    const int from = __ldcg(src + i), to = __ldcg(dst + i);
    if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages) {
      if (threadIdx.x == 0) raise_status(status, kStatusBadId);
      continue;
    }
    const uint8_t* a = p.base + pool * p.pool_stride + from * p.page_bytes;
    uint8_t* b = p.base + pool * p.pool_stride + to * p.page_bytes;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
      const int64_t off = static_cast<int64_t>(step) * kCopyBytes + (k * kCopyThreads + threadIdx.x) * 16;
      if (off < p.page_bytes) v[k] = __ldcs(reinterpret_cast<const uint4*>(a + off));
    }
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
      const int64_t off = static_cast<int64_t>(step) * kCopyBytes + (k * kCopyThreads + threadIdx.x) * 16;
      if (off < p.page_bytes) __stcs(reinterpret_cast<uint4*>(b + off), v[k]);
    }
  }
}

template <typename... Params, typename... Args>
bool launch_pdl(void (*kernel)(Params...), int grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, args...));
}

int copy_grid() { return 8 * device_info().num_sms; }

int launch_list_copy(const PagePool& p, const PagesWs& w, const int32_t* rank, unsigned* status, cudaStream_t s) {
  return launch_pdl(pages_copy_kernel, copy_grid(), kCopyThreads, s, p, static_cast<const int32_t*>(w.count), int64_t{0},
                    static_cast<const int32_t*>(w.src), static_cast<const int32_t*>(w.dst), rank, status)
             ? TQ1_OK
             : TQ1_ERR_CUDA;
}

}  // namespace

size_t pages_workspace_bytes(int64_t n_pages, int64_t n_seqs) {
  return (pages_words(n_pages, n_seqs) * sizeof(int32_t) + 255) & ~size_t(255);
}

int launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int64_t n, unsigned* status,
                      cudaStream_t s) {
  return launch_pdl(pages_copy_kernel, copy_grid(), kCopyThreads, s, p, static_cast<const int32_t*>(nullptr), n, src, dst,
                    static_cast<const int32_t*>(nullptr), status)
             ? TQ1_OK
             : TQ1_ERR_CUDA;
}

int launch_pages_resize(const PagePool& p, const int32_t* seqs, const int32_t* lens, int n, void* ws, unsigned* status,
                        cudaStream_t s) {
  const PagesWs w = split_ws(ws, p.n_pages);
  if (!launch_pdl(resize_kernel, 1, kPlanThreads, s, p, seqs, lens, n, w, status)) return TQ1_ERR_CUDA;
  return launch_list_copy(p, w, nullptr, status, s);
}

int launch_pages_fork(const PagePool& p, const int32_t* parents, const int32_t* children, int n, void* ws,
                      unsigned* status, cudaStream_t s) {
  const PagesWs w = split_ws(ws, p.n_pages);
  if (!launch_pdl(fork_kernel, 1, kPlanThreads, s, p, parents, children, n, w, status)) return TQ1_ERR_CUDA;
  return launch_list_copy(p, w, nullptr, status, s);
}

int launch_pages_compact(const PagePool& p, void* ws, unsigned* status, cudaStream_t s) {
  const PagesWs w = split_ws(ws, p.n_pages);
  const int chunks = (p.n_pages + kChunkPages - 1) / kChunkPages;
  if (!launch_pdl(compact_count_kernel, chunks, kPlanThreads, s, p, w)) return TQ1_ERR_CUDA;
  if (!launch_pdl(compact_plan_kernel, chunks, kPlanThreads, s, p, w)) return TQ1_ERR_CUDA;
  return launch_list_copy(p, w, w.rank, status, s);
}

}  // namespace tq1
