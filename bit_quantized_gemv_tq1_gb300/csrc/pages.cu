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
// Bound: the copies by HBM (each byte read and written once: 1.8 GB in pages
// of 32 KB at 6.8 TB/s, which is a plain copy's rate); the bookkeeping, a few
// thousand integers, by latency, which is why resize and fork do theirs in one
// CTA.  64 sequences that grow by 8 and shrink again, two calls: 11 us; 18
// beams freed and forked, 62 MB of copies: 20 us, half of it the copies.
#include "../../include/tq1.h"
#include "kv.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kChunkPages = 4 * kPlanThreads;  // pages of one compaction chunk
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;                             // 16-byte pieces per thread and step
constexpr int kStepVecs = kCopyThreads * kCopyVecs;      // of one step of a CTA

// Workspace: a header of 64 words, the copy list, and per-page / per-argument
// scratch.
struct PagesWs {
  int32_t* count;   // [0]: copies in the list; compaction: [1] live pages, [2] pages to move
  int32_t* src;     // [n_pages]
  int32_t* dst;     // [n_pages]
  int32_t* rank;    // [n_pages]   compaction: place of a moving page in the list
  int32_t* chunks;  // [ceil(n_pages / kChunkPages)] live pages per chunk
  int32_t* left;    // [n_seqs]    the page that argument i leaves for a copy of its own, or -1
};
__host__ __device__ inline size_t pages_words(int64_t n_pages, int64_t n_seqs) {
  return 64 + 3 * static_cast<size_t>(n_pages) + (n_pages + kChunkPages - 1) / kChunkPages + static_cast<size_t>(n_seqs);
}
inline PagesWs split_ws(void* ws, int64_t n_pages) {
  PagesWs w;
  w.count = static_cast<int32_t*>(ws);
  w.src = w.count + 64;
  w.dst = w.src + n_pages;
  w.rank = w.dst + n_pages;
  w.chunks = w.rank + n_pages;
  w.left = w.chunks + (n_pages + kChunkPages - 1) / kChunkPages;
  return w;
}

// Pages of `a` slots; any length up to the type's largest.
__device__ __forceinline__ int up(int a, const Divisor& b) { return a > 0 ? (a - 1) / b + 1 : 0; }
// Whether the last page of `a` > 0 slots is filled in part only.
__device__ __forceinline__ bool partly(int a, const Divisor& b) { return a / b * b.d != a; }

// This thread's four counts of the chunk of pages from `base` on; pages past
// the end are in use.
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int n_pages, int base) {
  const int p = base + 4 * static_cast<int>(threadIdx.x);
  if (p + 3 < n_pages) return __ldcg(reinterpret_cast<const int4*>(refs + p));
  int4 r = make_int4(1, 1, 1, 1);
  if (p < n_pages) r.x = __ldcg(refs + p);
  if (p + 1 < n_pages) r.y = __ldcg(refs + p + 1);
  if (p + 2 < n_pages) r.z = __ldcg(refs + p + 2);
  return r;
}

// The lowest `want` free pages into `out`, ascending, by the whole CTA, which
// holds the first chunk's counts in `r`; the scan stops as soon as it has
// them.  Returns how many there were (<= want).
__device__ int find_free(const int32_t* refs, int n_pages, int want, int4 r, int32_t* out, int* s_warp) {
  int found = 0;
  for (int base = 0;;) {
    const int mine = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int total;
    int at = found + block_scan<kPlanThreads>(mine, s_warp, total) - mine;
    const int p = base + 4 * static_cast<int>(threadIdx.x);
    if (r.x == 0 && at++ < want) out[at - 1] = p;
    if (r.y == 0 && at++ < want) out[at - 1] = p + 1;
    if (r.z == 0 && at++ < want) out[at - 1] = p + 2;
    if (r.w == 0 && at++ < want) out[at - 1] = p + 3;
    found += total;
    base += kChunkPages;
    if (found >= want || base >= n_pages) break;
    r = load_refs(refs, n_pages, base);
  }
  __syncthreads();
  return min(found, want);
}

constexpr int kNear = 2048;  // page ids kept in shared memory; more go through the workspace

// Runs of table entries to be dealt with, one per argument of a group: the
// warps take them in turn, a lane an entry, so that the long rows of a few
// sequences are spread over the CTA.  `count` < 1: none.
struct Runs {
  int64_t from[kPlanThreads], to[kPlanThreads];
  int count[kPlanThreads];
};
template <typename F>
__device__ __forceinline__ void each_run(const Runs& runs, int n, F act) {
  for (int i = threadIdx.x >> 5; i < min(n, kPlanThreads); i += kPlanThreads / 32)
    if (runs.count[i] > 0) act(runs.from[i], runs.to[i], runs.count[i]);
}
// Entries table[from + lane + 32 j], four loads at once.
template <typename F>
__device__ __forceinline__ void each_entry(const int32_t* table, int64_t from, int count, F act) {
  for (int j = threadIdx.x & 31; j < count; j += 128) {
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = j + 32 * u < count ? table[from + j + 32 * u] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (j + 32 * u < count) act(j + 32 * u, id[u]);
  }
}

// The arguments are taken kPlanThreads at a time, a thread each.  Every value
// that does not wait for the call's own changes (lengths, last pages, the
// first chunk of counts) is read before the first barrier: the kernel's time
// is the number of loads that have to follow one another.

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
  __shared__ int32_t s_free[kNear];
  __shared__ int s_copies;
  __shared__ unsigned long long s_wanted;
  __shared__ Runs runs;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) s_copies = s_wanted = 0;
  // 1
  int s = -1, len = 0, want = 0, last = -1;  // of the last group of arguments: the only one, for up to kPlanThreads
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    int keep = 0, had = 0;
    s = last = -1;
    if (i < n) {
      s = seqs[i];
      want = lens[i];
      if (s < 0 || s >= p.n_seqs) {
        raise_status(status, kStatusBadId);
        s = -1;
      } else {
        len = max(p.kv_len[s], 0);
        had = up(len, p.page_size);
        if (want < 0 || up(want, p.page_size) > p.max_pages || had > p.max_pages) {
          raise_status(status, kStatusNoPages);
          s = -1;
          had = 0;
        } else {
          if (want > len && partly(len, p.page_size)) last = p.table[static_cast<int64_t>(s) * p.max_pages + had - 1];
          keep = min(had, up(want, p.page_size));
          if (want <= len) p.kv_len[s] = want;
        }
      }
    }
    runs.from[threadIdx.x] = static_cast<int64_t>(max(s, 0)) * p.max_pages + keep;
    runs.count[threadIdx.x] = had - keep;
    if (__syncthreads_or(keep < had)) {
      each_run(runs, n - base, [&](int64_t from, int64_t, int count) {
        each_entry(p.table, from, count, [&](int j, int id) {
          if (id >= 0 && id < p.n_pages)
            atomicSub(p.refs + id, 1);
          else
            raise_status(status, kStatusBadId);
          p.table[from + j] = -1;
        });
      });
      __syncthreads();
    }
  }
  // 2 to 4
  const int4 refs0 = load_refs(p.refs, p.n_pages, 0);
  int64_t dealt = 0;
  int found = 0;  // free pages found
  int32_t* ids = s_free;
  const bool one_group = n <= kPlanThreads;
  if (!one_group) {
    // One search finds the pages of all groups: as many as they may want.
    unsigned long long wanted = 0;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
      const int t = seqs[i];
      if (t < 0 || t >= p.n_seqs) continue;
      const int l = max(p.kv_len[t], 0), v = lens[i];
      if (v > l && up(v, p.page_size) <= p.max_pages) wanted += up(v, p.page_size) - up(l, p.page_size) + 1;
    }
    atomicAdd(&s_wanted, wanted);
    __syncthreads();
    const int most = static_cast<int>(min(s_wanted, static_cast<unsigned long long>(p.n_pages)));
    if (most > kNear) ids = w.rank;
    if (most > 0) found = find_free(p.refs, p.n_pages, most, refs0, ids, s_warp);
  }
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    if (!one_group) {
      s = last = -1;
      if (i < n) {
        s = seqs[i];
        want = lens[i];
        if (s < 0 || s >= p.n_seqs) {
          s = -1;
        } else {
          len = max(p.kv_len[s], 0);
          if (want < 0 || up(want, p.page_size) > p.max_pages || up(len, p.page_size) > p.max_pages) s = -1;
          if (s >= 0 && want > len && partly(len, p.page_size))
            last = p.table[static_cast<int64_t>(s) * p.max_pages + up(len, p.page_size) - 1];
        }
      }
    }
    const bool grows = s >= 0 && want > len;
    const bool shared = grows && last >= 0 && last < p.n_pages && __ldcg(p.refs + last) > 1;
    const int first = up(len, p.page_size) - shared, need = grows ? up(want, p.page_size) - first : 0;
    int total;
    const int64_t at = dealt + block_scan<kPlanThreads>(need, s_warp, total) - need;
    if (one_group && total > 0) {
      if (total > kNear) ids = w.rank;
      found = find_free(p.refs, p.n_pages, min(total, p.n_pages), refs0, ids, s_warp);
    }
    dealt += total;
    const bool fits = grows && at + need <= found;
    if (grows && !fits) raise_status(status, kStatusNoPages);
    const int64_t row = static_cast<int64_t>(max(s, 0)) * p.max_pages + first;
    if (fits) {
      p.kv_len[s] = want;
      if (shared) {
        const int k = atomicAdd(&s_copies, 1);
        w.src[k] = last;
        w.dst[k] = ids[at];
      }
    }
    // A shared page is let go when every group has looked at its count.
    if (one_group) {
      if (fits && shared) atomicSub(p.refs + last, 1);
    } else if (i < n) {
      w.left[i] = fits && shared ? last : -1;
    }
    // New pages: one by its thread, more by a warp.
    const int gets = fits ? need : 0;
    if (gets == 1) {
      const int id = ids[at];
      p.table[row] = id;
      p.refs[id] = 1;
    }
    runs.from[threadIdx.x] = at;
    runs.to[threadIdx.x] = row;
    runs.count[threadIdx.x] = gets > 1 ? gets : 0;
    if (__syncthreads_or(gets > 1)) {
      each_run(runs, n - base, [&](int64_t from, int64_t to, int count) {
        for (int j = threadIdx.x & 31; j < count; j += 32) {
          const int id = ids[from + j];
          p.table[to + j] = id;
          p.refs[id] = 1;
        }
      });
      __syncthreads();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; !one_group && i < n; i += kPlanThreads)
    if (w.left[i] >= 0) atomicSub(p.refs + w.left[i], 1);
  if (threadIdx.x == 0) w.count[0] = s_copies;
}

// children[i] becomes a copy of parents[i]: whole pages shared, a partly
// filled last page copied to the lowest free one.
__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const PagePool p, const int32_t* parents,
                                                            const int32_t* children, int n, PagesWs w, unsigned* status) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int32_t s_free[kNear];
  __shared__ int s_copies;
  __shared__ Runs runs;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) s_copies = 0;
  const int4 refs0 = load_refs(p.refs, p.n_pages, 0);
  const int most = min(n, p.n_pages);  // a fork takes one page at most
  int32_t* ids = most <= kNear ? s_free : w.rank;
  const int have = find_free(p.refs, p.n_pages, most, refs0, ids, s_warp);
  int dealt = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    int s = -1, c = -1, len = 0;
    if (i < n) {
      s = parents[i];
      c = children[i];
      if (s < 0 || s >= p.n_seqs || c < 0 || c >= p.n_seqs || p.kv_len[c] != 0) {
        raise_status(status, kStatusBadId);
        s = -1;
      } else {
        len = p.kv_len[s];
        if (len <= 0 || up(len, p.page_size) > p.max_pages) s = -1;
      }
    }
    const int full = s >= 0 ? len / p.page_size : 0;
    const bool part = s >= 0 && partly(len, p.page_size);
    const int64_t from = static_cast<int64_t>(max(s, 0)) * p.max_pages, to = static_cast<int64_t>(max(c, 0)) * p.max_pages;
    const int last = part ? p.table[from + full] : -1;
    int total;
    const int at = dealt + block_scan<kPlanThreads>(part, s_warp, total) - part;
    const bool fits = at + part <= have;
    if (s >= 0 && !fits) raise_status(status, kStatusNoPages);
    const int gets = s >= 0 && fits ? full : 0;
    if (s >= 0 && fits) {
      p.kv_len[c] = len;
      if (part) {
        const int id = ids[at];
        if (last >= 0 && last < p.n_pages) {
          const int k = atomicAdd(&s_copies, 1);
          w.src[k] = last;
          w.dst[k] = id;
        } else {
          raise_status(status, kStatusBadId);
        }
        p.table[to + full] = id;
        p.refs[id] = 1;
      }
    }
    runs.from[threadIdx.x] = from;
    runs.to[threadIdx.x] = to;
    runs.count[threadIdx.x] = gets;
    __syncthreads();
    each_run(runs, n - base, [&](int64_t a, int64_t b, int count) {
      each_entry(p.table, a, count, [&](int j, int id) {
        p.table[b + j] = id;
        if (id >= 0 && id < p.n_pages)
          atomicAdd(p.refs + id, 1);
        else
          raise_status(status, kStatusBadId);
      });
    });
    __syncthreads();
    dealt += total;
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

// Up to kOwnCount chunks every CTA counts all of them itself (the counts come
// from L2, all loads at once), which is quicker than a kernel before this one;
// a thread's part of a chunk is four bits.
constexpr int kOwnCount = 16;

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagePool p, PagesWs w) {
  __shared__ int s_warp[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = gridDim.x, me = blockIdx.x, tid = threadIdx.x;
  int L, before_me, below, r[4], t;  // pages in use; those in chunks before this one; those below L
  if (chunks <= kOwnCount) {
    uint64_t bits = 0;
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
      (void)load_live4(p.refs, p.n_pages, c * kChunkPages + 4 * tid, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) bits |= static_cast<uint64_t>(r[i] > 0) << (4 * c + i);
    }
    (void)block_scan<kPlanThreads>(__popcll(bits), s_warp, L);
    (void)block_scan<kPlanThreads>(__popcll(bits & ((1ull << (4 * me)) - 1)), s_warp, before_me);
    const int cl = L / kChunkPages;  // L's chunk; past the last one when every page is in use
    uint64_t low = ~0ull;
    if (cl < kOwnCount) {
      const int in = min(max(L - cl * kChunkPages - 4 * tid, 0), 4);
      low = ((1ull << (4 * cl)) - 1) | (((1ull << in) - 1) << (4 * cl));
    }
    (void)block_scan<kPlanThreads>(__popcll(bits & low), s_warp, below);
  } else {
    const int v = tid < chunks ? __ldcg(w.chunks + tid) : 0;
    (void)block_scan<kPlanThreads>(v, s_warp, L);
    (void)block_scan<kPlanThreads>(tid < me ? v : 0, s_warp, before_me);
    const int cl = L / kChunkPages;
    (void)block_scan<kPlanThreads>(tid < cl ? v : 0, s_warp, below);
    if (L % kChunkPages != 0) {
      const int p0 = cl * kChunkPages + 4 * tid;
      (void)load_live4(p.refs, p.n_pages, p0, r);
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += p0 + i < L && r[i] > 0;
      (void)block_scan<kPlanThreads>(n, s_warp, t);
      below += t;
    }
  }
  const int p0 = me * kChunkPages + 4 * tid;
  const int live = load_live4(p.refs, p.n_pages, p0, r);
  int rank = before_me + block_scan<kPlanThreads>(live, s_warp, t) - live;  // pages in use before p0
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
  if (me == 0 && tid == 0) {
    w.count[0] = L - below;
    w.count[1] = L;
  }
}

// ---------------------------------------------------------------- copies --
// Every page of the list in every pool, in steps of 32 KB dealt to the CTAs in
// order; and, after a compaction plan, the tables' and counts'
// renaming, which touches nothing that is copied.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagePool p, const int32_t* count, int64_t n_fixed,
                                                                  const int32_t* src, const int32_t* dst,
                                                                  const int32_t* rank, unsigned* status) {
  pdl_launch_dependents();  // one wave: the next call's plan may start and wait
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
  // A step of a CTA is 32 KB of one page, or as many whole pages as that
  // holds: every thread has kCopyVecs loads in flight either way, and the
  // grid can be small (two CTAs an SM), which is what an empty list costs.
  const int page_vecs = static_cast<int>(p.page_bytes / 16), n32 = static_cast<int>(n);
  const int per_page = (page_vecs + kStepVecs - 1) / kStepVecs;  // steps of a page
  const int per_step = per_page > 1 ? 1 : kStepVecs / page_vecs;  // pages of a step
  const int64_t pages = n * p.n_pools, all = (pages + per_step - 1) / per_step * per_page;
  uint4 v[kCopyVecs];
  for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
    const int64_t first = u / per_page * per_step, pool0 = first / n;
    const int i0 = static_cast<int>(first - pool0 * n);
    if (per_step == 1) {
      const int from = src[i0], dest = dst[i0];
      if (from < 0 || from >= p.n_pages || dest < 0 || dest >= p.n_pages) {
        if (threadIdx.x == 0) raise_status(status, kStatusBadId);
        continue;
      }
      const int skip = static_cast<int>(u % per_page) * kStepVecs + threadIdx.x;
      uint8_t* const base = p.base + pool0 * p.pool_stride + static_cast<int64_t>(skip) * 16;
      const uint4* a = reinterpret_cast<const uint4*>(base + from * p.page_bytes);
      uint4* b = reinterpret_cast<uint4*>(base + dest * p.page_bytes);
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k)
        if (skip + k * kCopyThreads < page_vecs) v[k] = __ldcs(a + k * kCopyThreads);
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k)
        if (skip + k * kCopyThreads < page_vecs) __stcs(b + k * kCopyThreads, v[k]);
    } else {
      uint4* to[kCopyVecs];
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k) {
        const int at = k * kCopyThreads + static_cast<int>(threadIdx.x), sub = at / page_vecs;
        to[k] = nullptr;
        if (sub >= per_step || first + sub >= pages) continue;
        const int more = (i0 + sub) / n32, i = i0 + sub - more * n32;
        const int from = src[i], dest = dst[i];
        if (from < 0 || from >= p.n_pages || dest < 0 || dest >= p.n_pages) {
          raise_status(status, kStatusBadId);
          continue;
        }
        uint8_t* const base = p.base + (pool0 + more) * p.pool_stride + (at - sub * page_vecs) * 16;
        v[k] = __ldcs(reinterpret_cast<const uint4*>(base + from * p.page_bytes));
        to[k] = reinterpret_cast<uint4*>(base + dest * p.page_bytes);
      }
#pragma unroll
      for (int k = 0; k < kCopyVecs; ++k)
        if (to[k]) __stcs(to[k], v[k]);
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

int copy_grid() { return 2 * device_info().num_sms; }

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
  if (chunks > kOwnCount && !launch_pdl(compact_count_kernel, chunks, kPlanThreads, s, p, w)) return TQ1_ERR_CUDA;
  if (!launch_pdl(compact_plan_kernel, chunks, kPlanThreads, s, p, w)) return TQ1_ERR_CUDA;
  return launch_list_copy(p, w, w.rank, status, s);
}

}  // namespace tq1
