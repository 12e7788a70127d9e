// sample.cu -- the next token of each row of logits.
//
// Order a row's tokens by logit, the larger first, equal ones by index.  With
// w_i = exp((l_i - max) / T) the kept tokens are the shortest of three
// prefixes of that order: the first top_k; the shortest whose mass is at least
// top_p times the mass of the first top_k; the tokens with w >= min_p.  The
// token is the first whose prefix's mass exceeds u times the mass kept.  So
// everything is one question, asked up to three times: where does a count or
// a mass, summed in this order, reach a target?
//
// No sort of the vocabulary.  A first pass finds the largest logit, and a
// threshold that about as many tokens reach as will be needed; a second lists
// those tokens (and adds up all masses, by bins of (max - l) / T, where the mass
// of everything is asked for).  The list is sorted, and mostly every question
// has its answer there.  Where it has not, the masses (or counts) by bin say in
// which bin the target lies, 1/64 octave of weight; that bin's tokens are listed
// and sorted, together with those of the bins that the pick can be in, since
// where what is kept ends is known to a bin.  Bins of more than 1024 tokens are
// cut by the bits of their keys, down to a single value, whose tokens are
// counted off in index order.
//
// Sums: weights are integers in units of 2^-44, formed to within 2^-33 (the
// exponent in two fp32 parts, a table of 256 powers and a cubic), so masses
// add up exactly whatever the order, the token does not depend on how the row
// is divided, and a token changes only where u lands that near to a border.
// Less would not do: a row may have 2^19 borders.
//
// A row is read by a cluster of one to eight CTAs, as many as find room side by
// side with the rows there are; CTA 0 leads: it holds the merged masses and the
// list, and one thread of it decides what all do next.  Most code here runs once
// a row, and the time of a row is largely that of fetching it and of waiting for
// one another: one row of 131072 takes 3.7 us where the largest is asked for,
// 12.9 for a top_k of 50, 35.5 for a top_p of 0.95 with a wide nucleus.  Many
// rows are bound by instructions: a pass that adds up masses has some 40 a
// token (64 rows of 131072 in 63 us, 512 of 32000 in 95, and 5.5 for the largest, 6 TB/s).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/tq1.h"
#include "kv.cuh"
#include "step_internal.h"
#include "tq1_device.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kCuts = 2048;            // bins of a window (64 an octave of weight), parts of a range of keys
constexpr int kWindows = 2;            // windows of 32 octaves
constexpr uint32_t kNoBin = 0xffffffffu;
constexpr int kMostBits = 62;          // octaves that are told apart; what lies beyond is in the last bin
constexpr int kList = 1024;
// Tokens a list begins with, about, where no top_k says how many; a sixteenth of
// a short row, up to half as many as a CTA has threads (16 rows of 4000 with a
// top_p of 0.95 take 0.57 of the time that they take with 64; one row of 131072
// takes 1.02 times its time with 256, 152 rows of 16000 1.04).
constexpr int kWanted = 64;
constexpr int kShortRow = 16384;
// The largest top_k that begins with a list (400 of 131072 15.7 us, by bins 30.0;
// 600 34.1, since the list that was aimed at is often too long, and 30.3).
constexpr int kMostWanted = 400;
constexpr int kUnit = 44;              // weights in units of 2^-44
constexpr u64 kOne = u64{1} << kUnit;
constexpr int kMaxCluster = 8;
constexpr int kQueue = 2 * kList;      // groups that a pass has found and not looked at yet
constexpr int kBuckets = 256;          // of a list's tokens, by key

// What a pass does with the tokens of a range, or with all.
enum : int {
  kByKey = 1,    // the range is one of keys, else of bins
  kWeigh = 2,    // all: weights of `threshold` and more are added up
  kMasses = 4,   // range: masses by bin, or by part
  kCounts = 8,   // range: counts too
  kMerge = 16,   // the CTAs' masses and counts are added up in the leader
  kGather = 32,  // range: to the list
  kRange = 64,   // range: smallest and largest key
  kTally = 128,  // range: how many in each CTA
  kFind = 256,   // the nth token of the range in one CTA
  kDone = 512,
  kTop = 1024    // tokens from `lo` on: to the list
};

struct Command {
  int flags;
  uint32_t origin, span;  // range: [origin, origin + span]
  uint32_t second;        // kGather of bins: a bin that is gathered too
  int shift;              // parts of a range of keys: (key - origin) >> shift
  float lo;               // kTop
  float mid[2], half[2];  // logits that may be in the range are at most half from mid; and those of the second bin
  u64 threshold;          // kWeigh
  int rank, nth;          // kFind
};

// What the passes add up, in the leader's shared memory.
struct Result {
  u64 mass;    // sum of the pass
  unsigned n;  // tokens gathered
  uint32_t kmin, kmax;
  int found;   // kFind: the token, plus one; kGather: how many of n are of the second bin alone (and kmin their smallest key)
  unsigned tally[kMaxCluster];
};

// Differences are formed of halves, so that they stay finite.
struct Scale {
  float max;      // half the largest logit
  float c, c_lo;  // 2 log2(e) / T in two parts
};

// This CTA's part of a row.
struct Part {
  const void* p;
  int v;       // tokens
  int off;     // of the row's first token in its 16-byte group
  int j0, j1;  // this CTA's groups
  int rank, ranks;
  bool top;    // there are +inf: they are all equal, the others nothing
};

// What the leader's threads do next, together.
enum : int {
  kPass,    // with the other CTAs
  kOrder,   // the list
  kSearch,  // the masses by bin, or by part
  kLookUp,  // the target in the list
  kAbove,   // the mass of the list's tokens that weigh enough
  kEnd
};

// What one thread of the leader decides by.
struct State {
  int act, at;  // what to do next, and where to go on deciding then
  bool leave;   // the other CTAs are not needed any more
  bool last;    // what is done next is the last
  int question;  // 0: where the count reaches top_k, 1: the mass top_p of that, 2: the mass u of what is kept
  bool by_mass;
  u64 target;
  // The list.
  int n;          // its tokens
  bool whole;     // it begins with the row's first token
  bool complete;  // and holds every token that can be taken
  bool ordered;
  u64 in_list;    // the mass up to its end
  u64 before, skipped;  // the mass and the tokens before it
  int picks;      // so many of its tokens surround the pick, then `gap` of mass is missing
  u64 gap;
  uint32_t split; // the smallest key behind the gap
  u64 kept;       // the mass of what is kept so far
  bool any;       // that is known
  bool gone;      // the other CTAs have left
  // The search.
  int window;     // whose masses and counts the leader holds (merged), or -1
  bool first;     // the CTAs hold the first window's masses, to be merged
  bool found, by_key, pair, many;
  int by_bin;         // what lies before this bin is searched for, if any
  int i, shift;
  u64 mass0, count0;  // before the parts in shared memory
  u64 all_mass, all_count;
  u64 targets[2];
  int bin[2];
  u64 count_before[2], mass_before[2];
  u64 tokens;
  uint32_t klo, khi, b0, b1, pick_bin;
  u64 start, nth, one;
  // The answer.
  u64 mass_at, weight_at;
  int token;          // -1: not found, which only logits that change under the call can bring about
};

// A row's filters.
struct Filters {
  float temperature, top_p, min_p, u;
  int top_k;
  bool by_k, by_p, by_m, greedy;
};

// All that is the same for a CTA's threads and outlives a pass lives here: on
// the threads' stacks it would be 512 copies, more than the cache holds.
struct Shared {
  // Masses (low and high words) and counts by bin or by part of a range of
  // keys: this CTA's, in the leader the row's once they are merged.
  unsigned low[kCuts], high[kCuts], count[kCuts];
  u64 stage[kList];       // what this CTA gathers
  u64 list[kList];        // leader: the gathered tokens
  union {
    u64 prefix[kList];    // leader: masses up to and with each, in the row's order
    int queue[kQueue];
  };
  int place[kList];       // leader: how many of the list come before each token
  int pow[256];           // 2^30 2^(-i/256)
  u64 part[2][16];
  unsigned n_stage, at_stage, n_queue, n_second, second_min;
  int bucket[kBuckets + 1];
  float red[16];
  uint32_t red_low[16], red_high[16];
  int red_at[16];
  float best[kMaxCluster], least[kMaxCluster];  // of each CTA: its largest logit, the lower end of its list
  int best_at[kMaxCluster];
  Part row;
  // Read once by each CTA, for its part of the list's threshold, and by the
  // leader for all: should they change under the call, all still do the same.
  Filters own, filters;
  Scale scale;
  Command cmd;
  Result sum;
  State state;  // leader
  Command next;
};

__device__ __forceinline__ Shared& shared() {
  extern __shared__ __align__(16) uint8_t smem[];
  return *reinterpret_cast<Shared*>(smem);
}
__device__ __forceinline__ Shared& shared_of(int rank) { return *cg::this_cluster().map_shared_rank(&shared(), rank); }

__device__ __forceinline__ void sync_row(int ranks) {
  if (ranks == 1) __syncthreads();
  else cg::this_cluster().sync();
}

// -------------------------------------------------------------- weights --
// 2^30 2^(-i/256): products of the roots 2^(-1/2) .. 2^(-1/256).
struct Powers {
  int w[256];
};
constexpr Powers make_powers() {
  const double roots[8] = {0.70710678118654752440, 0.84089641525371454303, 0.91700404320467123174, 0.95760328069857364693,
                           0.97857206208770013450, 0.98922801319397548412, 0.99459942348363317565, 0.99729605608547012625};
  Powers p{};
  for (int i = 0; i < 256; ++i) {
    double v = 1073741824.0;
    for (int b = 0; b < 8; ++b)
      if (i & (128 >> b)) v *= roots[b];
    p.w[i] = static_cast<int>(v + 0.5);
  }
  return p;
}
__device__ const Powers kPowers = make_powers();

// Order by logit: the smaller key is the larger logit.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key : (~key & 0x7FFFFFFFu));
}

// p = (max - l) log2(e) / T in two parts: p (at most 62: from 45 on nothing
// is left) and what rounding lost, and k, the integer nearest to 256 p.  The
// bins are those of k, 64 an octave.
struct Exponent {
  float p, p_lo, biased;
  int k;
};
__device__ __forceinline__ Exponent exponent_of(const Scale& s, float l) {
  const float h = 0.5f * l, d = s.max - h;
  const float t = d - s.max;
  const float d_lo = (s.max - (d - t)) + (-h - t);  // what the difference lost (two-sum)
  Exponent e;
  const float full = d * s.c;
  e.p = fminf(full, static_cast<float>(kMostBits));
  e.p_lo = fmaf(d, s.c, -full) + fmaf(d, s.c_lo, d_lo * s.c);  // NaN where nothing is left: it does not matter
  e.biased = fmaf(e.p, 256.0f, 12582912.0f);                   // 1.5 2^23 + k
  e.k = __float_as_int(e.biased) & 0x3FFFFF;
  return e;
}
__device__ __forceinline__ uint32_t bin_of(int k) { return static_cast<uint32_t>(k) >> 2; }

// 2^31 2^-(p mod 1): 2^-(r + p_lo) - 1 = -z + z^2/2 - z^3/6 with r = p - k/256
// (exact, |r| <= 1/512), z = (r + p_lo) ln 2 <= 0.00136: off by 2^-33.
__device__ __forceinline__ unsigned mantissa_of(const int* pow, const Exponent& x) {
  const float r = fmaf(x.biased - 12582912.0f, -0.00390625f, x.p);
  const float z = fmaf(x.p_lo, 0.69314718f, r * 0.69314718f);
  const float e = z * fmaf(z, fmaf(z, -0.16666667f, 0.5f), -1.0f);
  const int half = pow[x.k & 255];
  return 2 * half + __mulhi(half, __float2int_rn(e * 8589934592.0f));
}
// m 2^-down, rounded.
__device__ __forceinline__ unsigned shifted(unsigned m, int down) {
  return __funnelshift_rc(m + ((1u << (down & 31)) >> 1), 0u, down);
}
// 2^44 exp((l - max) / T) as an integer.
__device__ __forceinline__ u64 weight_of(const int* pow, const Exponent& x) {
  const unsigned m = mantissa_of(pow, x);
  const int down = (x.k >> 8) - 13;
  return down > 0 ? shifted(m, down) : static_cast<u64>(m) << -down;
}
__device__ __forceinline__ u64 weight_of(const int* pow, const Scale& s, float l) { return weight_of(pow, exponent_of(s, l)); }

// floor(f z), or ceil(f z), for f in (0, 1).
__device__ __noinline__ u64 part_of(u64 z, float f, bool up) {
  const unsigned bits = __float_as_uint(f), e = bits >> 23;
  const u64 mant = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  int sh = 150 - static_cast<int>(e ? e : 1);  // f = mant 2^-sh, sh >= 24
  u64 hi = __umul64hi(z, mant), lo = z * mant;
  bool rest = false;
  while (sh > 0) {  // 63 bits at a time
    const int n = min(sh, 63);
    rest |= (lo << (64 - n)) != 0;
    lo = (lo >> n) | (hi << (64 - n));
    hi >>= n;
    sh -= n;
  }
  return lo + (up && rest);
}

// ---------------------------------------------------------------- blocks --
// Of every thread: the sum of v over the threads before it; `all` the sum over all.
template <int N, int M>
__device__ __forceinline__ void block_before(u64 (&v)[M], u64 (&all)[M]) {
  Shared& sh = shared();
  constexpr int kWarps = N / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 own[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    own[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += x;
    }
    if (lane == 31) sh.part[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < M; ++i) {
    v[i] -= own[i];
    all[i] = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const u64 x = sh.part[i][w];
      all[i] += x;
      if (w < warp) v[i] += x;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ rows --
template <typename T, int N>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* p;
  int v;       // tokens
  int off;     // of the row's first token in its 16-byte group
  int j0, j1;  // this CTA's groups
  bool top;    // there are +inf: they are all equal, the others nothing

  __device__ __forceinline__ Row() {
    const Part& r = shared().row;
    p = static_cast<const T*>(r.p);
    v = r.v;
    off = r.off;
    j0 = r.j0;
    j1 = r.j1;
    top = r.top;
  }

  // NaN is never taken; -0 equals 0.
  __device__ __forceinline__ static float ordered(float l) { return l == l ? l + 0.0f : -INFINITY; }
  // Of a logit of the row, once: where there are +inf, a second time would find none.
  __device__ __forceinline__ float value(float l) const {
    return top ? (l == INFINITY ? 0.0f : -INFINITY) : ordered(l);
  }

  // The logits of a group, as they are.
  __device__ __forceinline__ static void unpack(const uint4& raw, float (&l)[kVec]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kVec == 4) {
        l[i] = __uint_as_float(w[i]);
      } else {
        const float2 two = unpack2<T>(w[i]);
        l[2 * i] = two.x;
        l[2 * i + 1] = two.y;
      }
    }
  }

  // A group; what lies outside the row is -inf.
  __device__ __forceinline__ uint4 load(int g) const {
    const int at = g * kVec - off;
    if (at >= 0 && at + kVec <= v) return *reinterpret_cast<const uint4*>(p + at);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kVec == 4) {
        w[i] = at + i >= 0 && at + i < v ? reinterpret_cast<const uint32_t*>(p)[at + i] : 0xFF800000u;
      } else {
        const uint32_t none = pack2<T>(-INFINITY, -INFINITY);
        const int c = at + 2 * i;
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        const uint32_t lo = c >= 0 && c < v ? q[c] : none & 0xFFFFu, hi = c + 1 >= 0 && c + 1 < v ? q[c + 1] : none >> 16;
        w[i] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  // look(g) for those groups g of this CTA's part for which fast(logits as
  // they are, g) holds, and for the row's ragged ends.
  template <typename Fast, typename Look>
  __device__ __forceinline__ void scan(Fast&& fast, Look&& look) const {
    constexpr int kAhead = 4;  // 16-byte loads a thread has in flight
    const int tid = threadIdx.x;
    const int f0 = off ? max(j0, 1) : j0, f1 = min(j1, (v + off) / kVec);  // whole groups
    const uint4* from = reinterpret_cast<const uint4*>(p - off);
    int end = -1;  // the first group, or the last, where it is not whole
    if (tid == 0 && f0 > j0 && j0 < j1) end = j0;
    if (tid == 1 && f1 < j1 && j0 < j1 && !(f0 > j0 && j1 - j0 == 1)) end = j1 - 1;
    int j = f0 + tid;
    do {
      uint4 raw[kAhead];
      unsigned hits = end >= 0 ? 1u << kAhead : 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (j + i * N < f1) raw[i] = from[j + i * N];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (j + i * N < f1) {
          float one[kVec];
          unpack(raw[i], one);
          if (fast(one, j + i * N)) hits |= 1u << i;
        }
      }
      while (hits) {
        const int i = __ffs(hits) - 1;
        hits &= hits - 1;
        look(i == kAhead ? end : j + i * N);
      }
      end = -1;
      j += kAhead * N;
    } while (j < f1);
  }

  // f(four logits) for this CTA's part of the row, as they are, but where there
  // are +inf their values; -inf where a thread has none.  Two groups are on their way while
  // two are worked on.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    const int tid = threadIdx.x;
    const int f0 = off ? max(j0, 1) : j0, f1 = min(j1, (v + off) / kVec);  // whole groups
    const uint4* from = reinterpret_cast<const uint4*>(p - off);
    const uint32_t low = kVec == 4 ? 0xFF800000u : pack2_none();
    const uint4 none = make_uint4(low, low, low, low);
    // The ragged ends go first, as two more groups of the first two threads.
    uint4 a = none, b = none;
    int j = f0 + tid;
    if (tid == 0 && f0 > j0 && j0 < j1) a = load(j0);
    if (tid == 1 && f1 < j1 && j0 < j1 && !(f0 > j0 && j1 - j0 == 1)) a = load(j1 - 1);
#pragma unroll 1
    for (;;) {
      uint4 c = none, d = none;
      if (j < f1) c = from[j];
      if (j + N < f1) d = from[j + N];
      work(a, f);
      work(b, f);
      if (j >= f1) break;
      a = c;
      b = d;
      j += 2 * N;
    }
  }
  __device__ __forceinline__ static uint32_t pack2_none() {
    if constexpr (kVec == 8) return pack2<T>(-INFINITY, -INFINITY);
    else return 0;
  }
  template <typename F>
  __device__ __forceinline__ void work(const uint4& raw, F&& f) const {
    float l[kVec];
    unpack(raw, l);
#pragma unroll
    for (int h = 0; h < kVec; h += 4) {
      float four[4] = {l[h], l[h + 1], l[h + 2], l[h + 3]};
      if (top) {
#pragma unroll
        for (int i = 0; i < 4; ++i) four[i] = value(four[i]);
      }
      f(four);
    }
  }
};

__device__ __forceinline__ void put(Shared& sh, uint32_t key, int at) {
  if (*static_cast<volatile unsigned*>(&sh.n_stage) > kList) return;  // too many: how many does not matter
  const unsigned i = atomicAdd(&sh.n_stage, 1u);
  if (i < kList) sh.stage[i] = (static_cast<u64>(key) << 32) | static_cast<uint32_t>(at);
}

// ---------------------------------------------------------------- passes --
// What sh.cmd says, by one CTA of the row's cluster.
template <typename T, int N>
__device__ __noinline__ void pass() {
  Shared& sh = shared();
  const int tid = threadIdx.x, flags = sh.cmd.flags, ranks = sh.row.ranks;
  if (tid == 0) {
    sh.n_stage = sh.n_queue = sh.n_second = 0;
    sh.second_min = 0xffffffffu;
  }
  if (flags & kMasses)
    for (int i = tid; i < kCuts; i += N) sh.low[i] = sh.high[i] = sh.count[i] = 0;
  __syncthreads();
  const uint32_t origin = sh.cmd.origin, span = sh.cmd.span;
  u64 mine = 0;
  if (flags & (kWeigh | kMasses)) {
    const Row<T, N> row;
    const Scale s = sh.scale;
    const int shift = sh.cmd.shift;
    row.each([&](const float (&l)[4]) {
      // Weights are below 2^32 but for the likeliest tokens'.  What cannot be
      // taken, NaN too, has p = 62 and weighs nothing.
      unsigned lo[4], hi[4];
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Exponent e = exponent_of(s, l[i]);
        const unsigned m = mantissa_of(sh.pow, e);
        const int down = (e.k >> 8) - 13;
        lo[i] = shifted(m, down);
        hi[i] = 0;
        if (down <= 0) {
          lo[i] = m << -down;
          hi[i] = __funnelshift_l(m, 0u, -down);
        }
        x[i] = bin_of(e.k);
      }
      if (flags & kByKey) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = key_of(Row<T, N>::ordered(l[i]));
      }
      if (!(flags & kMasses)) {
        const u64 least = sh.cmd.threshold;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u64 w = (static_cast<u64>(hi[i]) << 32) | lo[i];
          mine += w >= least ? w : 0;
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mine += lo[i];
        x[i] -= origin;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (hi[i]) mine += static_cast<u64>(hi[i]) << 32;
        if (x[i] <= span) {
          const unsigned old = atomicAdd(&sh.low[x[i] >> shift], lo[i]);
          const unsigned more = hi[i] + (old + lo[i] < old ? 1u : 0u);
          if (more) atomicAdd(&sh.high[x[i] >> shift], more);
          if ((flags & kCounts) && l[i] > -INFINITY) atomicAdd(&sh.count[x[i] >> shift], 1u);
        }
      }
    });
  }
  unsigned seen = 0;
  uint32_t kmin = 0xffffffffu, kmax = 0;
  if (flags & (kGather | kTop | kRange | kTally)) {
    const Row<T, N> row;
    const float lo = sh.cmd.lo, mid = sh.cmd.mid[0], half = sh.cmd.half[0];
    const uint32_t second = sh.cmd.second;
    auto look = [&](int at) {
      const float l = row.value(static_cast<float>(row.p[at]));
      const uint32_t k = key_of(l);
      bool in, other = false;
      if (flags & kTop) {
        in = row.top || l >= lo;
      } else {
        const uint32_t x = (flags & kByKey) ? k : bin_of(exponent_of(sh.scale, l).k);
        in = x - origin <= span;
        other = !in && x == second && !(flags & kByKey);
      }
      if (other && l != -INFINITY) {
        atomicAdd(&sh.n_second, 1u);
        atomicMin(&sh.second_min, k);
      }
      if ((in || other) && l != -INFINITY) {
        if (flags & (kGather | kTop)) put(sh, k, at);
        ++seen;
        kmin = min(kmin, k);
        kmax = max(kmax, k);
      }
    };
    row.scan(
        [&](const float (&one)[Row<T, N>::kVec], int) {
          auto nearest = [&](float to) {
            float m = fabsf(one[0] - to);  // NaN: another's
#pragma unroll
            for (int i = 1; i < Row<T, N>::kVec; ++i) m = fminf(m, fabsf(one[i] - to));
            return m;
          };
          if (nearest(mid) <= half) return true;
          return second != kNoBin && nearest(sh.cmd.mid[1]) <= sh.cmd.half[1];
        },
        [&](int g) {  // later, by all threads
          const unsigned i = atomicAdd(&sh.n_queue, 1u);
          if (i < kQueue) {
            sh.queue[i] = g;
          } else {
            const int at = g * Row<T, N>::kVec - row.off;
#pragma unroll 1
            for (int j = max(at, 0); j < min(at + Row<T, N>::kVec, row.v); ++j) look(j);
          }
        });
    __syncthreads();
    const int many = min(sh.n_queue, static_cast<unsigned>(kQueue)) * Row<T, N>::kVec;
#pragma unroll 1
    for (int i = tid; i < many; i += N) {
      const int at = sh.queue[i / Row<T, N>::kVec] * Row<T, N>::kVec - row.off + i % Row<T, N>::kVec;
      if (at >= 0 && at < row.v) look(at);
    }
  }
  Shared& lead = ranks == 1 ? sh : shared_of(0);
  if (flags & kWeigh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((tid & 31) == 0 && mine) atomicAdd(&lead.sum.mass, mine);
  }
  if (flags & (kRange | kTally)) {
    seen = __reduce_add_sync(0xffffffffu, seen);
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if ((tid & 31) == 0) {
      atomicAdd(&lead.sum.tally[sh.row.rank], seen);
      atomicMin(&lead.sum.kmin, kmin);
      atomicMax(&lead.sum.kmax, kmax);
    }
  }
  if (flags & (kGather | kTop)) {  // what this CTA gathered goes to the leader's list
    __syncthreads();
    const unsigned n = min(sh.n_stage, kList + 1u);  // one more than there is room for: too many
    if (tid == 0) {
      sh.at_stage = n ? atomicAdd(&lead.sum.n, n) : 0;
      if (sh.n_second) {
        atomicAdd(&lead.sum.found, static_cast<int>(sh.n_second));
        atomicMin(&lead.sum.kmin, sh.second_min);
      }
    }
    __syncthreads();
    const unsigned at = sh.at_stage;
    for (unsigned i = tid; i < min(n, static_cast<unsigned>(kList)); i += N)
      if (at + i < kList) lead.list[at + i] = sh.stage[i];
  }
  if (flags & kMerge) {
    sync_row(ranks);
    if (ranks > 1) {  // each CTA a part of the bins, read from all the others
      const int per = (kCuts + ranks - 1) / ranks;
      for (int i = sh.row.rank * per + tid; i < min(kCuts, (sh.row.rank + 1) * per); i += N) {
        u64 m = 0;
        unsigned n = 0;
#pragma unroll 4
        for (int r = 0; r < ranks; ++r) {
          const Shared& o = shared_of(r);
          m += (static_cast<u64>(o.high[i]) << 32) + o.low[i];
          n += o.count[i];
        }
        lead.low[i] = static_cast<unsigned>(m);
        lead.high[i] = static_cast<unsigned>(m >> 32);
        lead.count[i] = n;
      }
    }
  }
  if ((flags & kFind) && sh.cmd.rank == sh.row.rank) {  // in index order
    const Row<T, N> row;
    int left = sh.cmd.nth;  // 1-based
    const int from = max(0, row.j0 * Row<T, N>::kVec - row.off), to = min(row.v, row.j1 * Row<T, N>::kVec - row.off);
    for (int base = from; base < to; base += N) {
      const int at = base + tid;
      float l = -INFINITY;
      if (at < to) l = row.value(static_cast<float>(row.p[at]));
      const bool hit = l != -INFINITY && key_of(l) == origin;
      const uint32_t b = __ballot_sync(0xffffffffu, hit);
      if ((tid & 31) == 0) sh.red_at[tid >> 5] = __popc(b);
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll 1
      for (int w = 0; w < N / 32; ++w) {
        if (w < (tid >> 5)) before += sh.red_at[w];
        all += sh.red_at[w];
      }
      before += __popc(b & ((1u << (tid & 31)) - 1u));
      if (hit && before + 1 == left) lead.sum.found = at + 1;
      __syncthreads();
      if (all >= left) break;
      left -= all;
    }
  }
  sync_row(ranks);
}

// The middle of [lo, hi], and what the farthest from it are off, with room for
// the rounding of both and of a difference from it (halves of subnormal values, too,
// of which two steps are lost at most); without bounds 0 and infinity.
__device__ __forceinline__ void middle_of(float lo, float hi, float& mid, float& half) {
  mid = 0.5f * lo + 0.5f * hi;
  half = 0.5f * hi - 0.5f * lo + 2.4e-7f * (fabsf(lo) + fabsf(hi)) + 1.1e-44f;
  if (!(half < INFINITY)) {
    mid = 0.0f;
    half = INFINITY;
  }
}
// Of the logits of some bins, and somewhat more than rounding may add.
__device__ __forceinline__ void middle_of_bins(const Scale& s, uint32_t first, uint32_t last, float& mid, float& half) {
  const float far = (4.0f * last + 4.0f) / (256.0f * s.c), near = (4.0f * first - 1.0f) / (256.0f * s.c);
  const float slack = 1e-6f * (fabsf(s.max) + far);
  middle_of(2.0f * (s.max - far - slack), 2.0f * (s.max - near + slack), mid, half);
}

// Asks for a pass of all CTAs.
__device__ __noinline__ int ask(int flags, uint32_t origin, uint32_t span, int shift, u64 threshold = 0, int rank = 0, int nth = 0,
                                uint32_t second = kNoBin) {
  Shared& sh = shared();
  for (int i = 0; i < kMaxCluster; ++i) sh.sum.tally[i] = 0;
  sh.sum.mass = 0;
  sh.sum.n = 0;
  sh.sum.kmin = 0xffffffffu;
  sh.sum.kmax = 0;
  sh.sum.found = 0;
  Command c = {flags, origin, span, second, shift, 0.0f, {0.0f, 0.0f}, {INFINITY, INFINITY}, threshold, rank, nth};
  if (sh.row.top) {
    // All that is +inf.
  } else if (flags & kByKey) {
    middle_of(logit_of(origin + span), logit_of(origin), c.mid[0], c.half[0]);
  } else if (sh.scale.c > 0.0f && origin + span < kMostBits * 64) {
    middle_of_bins(sh.scale, origin, origin + span, c.mid[0], c.half[0]);
    if (second != kNoBin) middle_of_bins(sh.scale, second, second, c.mid[1], c.half[1]);
  }
  sh.next = c;
  return kPass;
}

// The others may leave: nothing more is asked of them.  They are not waited for.
__device__ __noinline__ void dismiss(int ranks) {
  __syncthreads();
  if (threadIdx.x < ranks) shared_of(threadIdx.x).cmd.flags = kDone;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

// The list's n tokens: their places (how many come before each) and the masses
// up to and with each place (prefix), the mass before the list included.
// At the place `picks` a gap of mass lies before the token that is not the
// list's.  A token is compared with those of its bucket
// only: buckets are even parts of the range of (key, index), of which a type's
// `unused` low key bits are left out, so that equal logits fall apart by index,
// and what lies between the two parts of a list with a gap.
template <int N>
__device__ __noinline__ void order(int unused) {
  Shared& sh = shared();
  const int n = sh.state.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t split = sh.state.split;
  uint32_t first = 0xffffffffu, last = 0, end = split;
#pragma unroll 1
  for (int i = tid; i < n; i += N) {
    const uint32_t k = static_cast<uint32_t>(sh.list[i] >> 32);
    first = min(first, k);
    if (k < split) last = max(last, k);
    else end = max(end, k);
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  end = __reduce_max_sync(0xffffffffu, end);
  if (lane == 0) {
    sh.red_low[warp] = first;
    sh.red_high[warp] = last;
    sh.red_at[warp] = static_cast<int>(end);
  }
  if (tid < kBuckets) sh.bucket[tid] = 0;
  __syncthreads();
  first = __reduce_min_sync(0xffffffffu, sh.red_low[lane & (N / 32 - 1)]);
  last = __reduce_max_sync(0xffffffffu, sh.red_high[lane & (N / 32 - 1)]);
  end = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(sh.red_at[lane & (N / 32 - 1)]));
  const int bits = 32 - __clz(sh.row.v - 1 | 1);  // of an index
  const uint32_t rest = last < first ? 0 : ((last - first) >> unused) + 1;  // where the part behind the gap begins
  auto place_of = [&](uint32_t k) { return k < split ? (k - first) >> unused : rest + ((k - split) >> unused); };
  const int shift = max(0, 56 - __clzll((static_cast<u64>(place_of(max(last, end))) << bits) | ((u64{1} << bits) - 1)));
  auto bucket_of = [&](u64 token) {
    return static_cast<int>(((static_cast<u64>(place_of(static_cast<uint32_t>(token >> 32))) << bits) | static_cast<uint32_t>(token)) >> shift);
  };
#pragma unroll 1
  for (int i = tid; i < n; i += N)
    sh.place[i] = atomicAdd(&sh.bucket[bucket_of(sh.list[i])], 1);
  __syncthreads();
  if (warp == 0) {  // where each bucket begins
    constexpr int kPer = kBuckets / 32;
    int own[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      own[i] = sh.bucket[lane * kPer + i];
      sum += own[i];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sh.bucket[lane * kPer + i] = before;
      before += own[i];
    }
    if (lane == 31) sh.bucket[kBuckets] = before;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < n; i += N) {
    const u64 own = sh.list[i];
    sh.stage[sh.bucket[bucket_of(own)] + sh.place[i]] = own;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < n; i += N) {
    const u64 own = sh.list[i];
    const int b = bucket_of(own);
    const int from = sh.bucket[b], to = sh.bucket[b + 1];
    int place = from;
#pragma unroll 4
    for (int j = from; j < to; ++j) place += sh.stage[j] < own;
    sh.place[i] = place;
    sh.prefix[place] = weight_of(sh.pow, sh.scale, logit_of(static_cast<uint32_t>(own >> 32)));
  }
  __syncthreads();
  u64 upto = sh.state.before;
  const u64 gap = sh.state.gap;
  const int picks = sh.state.picks;
#pragma unroll 1
  for (int from = 0; from < n; from += N) {
    const int at = from + tid;
    const u64 own = at < n ? sh.prefix[at] + (at == picks ? gap : 0) : 0;
    u64 v[1] = {own}, all[1];
    block_before<N>(v, all);
    if (at < n) sh.prefix[at] = upto + v[0] + own;
    upto += all[0];
  }
  if (tid == 0) sh.state.in_list = upto;
  __syncthreads();
}

// The parts of those in shared memory at which the count or the mass reaches
// each target, and what lies before them.
template <int N>
__device__ __noinline__ void search() {
  Shared& sh = shared();
  State& s = sh.state;
  constexpr int kPer = kCuts / N;
  // A warp's parts lie behind one another, a lane's kPer of them too; lanes
  // read theirs in different orders, so that no eight of them meet in a bank.
  const int b0 = threadIdx.x * kPer, turn = threadIdx.x / (32 / kPer);
  const bool by_mass = s.by_mass || s.pair;
  u64 v[2] = {0, 0}, all[2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + ((i + turn) & (kPer - 1));
    v[0] += (static_cast<u64>(sh.high[b]) << 32) + sh.low[b];
    v[1] += sh.count[b];
  }
  const u64 own = by_mass ? v[0] : v[1];
  block_before<N>(v, all);
  if (threadIdx.x == 0) {
    s.all_mass = all[0];
    s.all_count = all[1];
  }
  v[0] += s.mass0;
  v[1] += s.count0;
#pragma unroll 1
  for (int j = 0; j < (s.pair ? 2 : 1); ++j) {
    const u64 want = s.targets[j], had = by_mass ? v[0] : v[1];
    if (s.by_bin >= 0 ? s.by_bin / kPer == static_cast<int>(threadIdx.x) : (had < want && had + own >= want)) {
      u64 mass = v[0], count = v[1];
#pragma unroll 1
      for (int b = b0; b < b0 + kPer; ++b) {
        const u64 m = mass + (static_cast<u64>(sh.high[b]) << 32) + sh.low[b], c = count + sh.count[b];
        if (s.by_bin >= 0 ? b == s.by_bin : (by_mass ? m : c) >= want) {
          s.bin[j] = b;
          s.mass_before[j] = mass;
          s.count_before[j] = count;
          break;
        }
        mass = m;
        count = c;
      }
    }
  }
  __syncthreads();
}

// w / z in fp32, what the conversions lost made good: one rounding.
__device__ __forceinline__ float ratio_of(u64 w, u64 z) {
  const float wh = __ull2float_rn(w), zh = __ull2float_rn(z);
  const float wl = __ll2float_rn(static_cast<long long>(w - __float2ull_rn(wh))), zl = __ll2float_rn(static_cast<long long>(z - __float2ull_rn(zh)));
  const float q = __fdiv_rn(wh, zh);
  return q + (fmaf(-q, zh, wh) + fmaf(-q, zl, wl)) / zh;
}

// The pick is where the mass reaches this.
__device__ __forceinline__ u64 pick_of(float u, u64 mass) {
  if (!(u < 1.0f)) return mass;  // NaN too
  return u > 0.0f ? min(mass, part_of(mass, u, false) + 1) : u64{1};
}

__device__ __forceinline__ u64 mass_of_bin(const Shared& sh, uint32_t b) { return (static_cast<u64>(sh.high[b]) << 32) + sh.low[b]; }

// About how many tokens a bin of the first window holds.
__device__ __forceinline__ float tokens_of_bin(const Shared& sh, uint32_t b) {
  return __ull2float_rn(mass_of_bin(sh, b)) * exp2f(static_cast<float>(b) * 0.015625f - kUnit);
}

// Whether the tokens of a few bins, and of one at or behind them, are for the list.
__device__ __forceinline__ bool fit(const Shared& sh, int first, int last, int other) {
  if (last - first >= 16) return false;
  float tokens = other > last ? tokens_of_bin(sh, other) : 0.0f;
  for (int b = first; b <= last && tokens <= kList; ++b) tokens += tokens_of_bin(sh, b);
  return tokens <= kList;
}

// The bin of a token that weighs w, or -1: behind the first window, or so near
// to a border that another rounding may find the next bin.
__device__ __forceinline__ int bin_of_weight(float w) {
  const float x = fmaxf(-64.0f * log2f(w), 0.0f) + 0.125f, in = x - floorf(x);
  return x < kCuts && in > 0.01f && in < 0.99f ? static_cast<int>(x) : -1;
}

// The gathered list holds the tokens of the bins around the pick, and of bin b1,
// before which `before` of mass and `tokens` tokens lie.
__device__ __forceinline__ void take_pair(const Shared& sh, State& s) {
  s.picks = static_cast<int>(sh.sum.n) - sh.sum.found;
  s.split = sh.sum.kmin;
  u64 end = s.mass_before[0];
  for (int b = s.bin[0]; b <= s.bin[1]; ++b) end += mass_of_bin(sh, b);
  const bool apart = static_cast<int>(s.b1) > s.bin[1];
  s.gap = apart ? s.before - end : 0;
  s.tokens = apart ? s.tokens - s.picks : s.count_before[0];
  s.before = s.mass_before[0];
}

// What the leader's threads do next: one thread decides, from the state, where
// all would hold a copy of it and spill it.  It goes on where it had left off:
// TQ1_DO leaves, and the next call comes back there.
#define TQ1_DO(what) \
  do {               \
    s.at = __LINE__; \
    return what;     \
    case __LINE__:;  \
  } while (0)
__device__ __noinline__ int decide() {
  Shared& sh = shared();
  State& s = sh.state;
  const Filters& f = sh.filters;
  s.leave = s.last = false;
  switch (s.at) {
    case 0:
      for (s.question = 0; s.question < 3; ++s.question) {
        if (s.question == 0 ? !f.by_k : s.question == 1 ? !f.by_p : false) continue;
        if (s.question == 2 && f.by_m) {
          // What weighs min_p of the largest or more.
          if (s.whole && !s.ordered) {
            if (s.complete) s.leave = !s.gone;
            s.gone |= s.leave;
            TQ1_DO(kOrder);
            s.ordered = true;
          }
          s.one = f.min_p < 1.0f ? max(u64{1}, part_of(kOne, f.min_p, true)) : kOne;
          // Of the list, where that holds all that is kept, or ends with less weight.
          if (s.whole && (s.complete || (s.any && s.kept <= s.in_list) ||
                          (s.n > 0 && s.in_list - (s.n > 1 ? sh.prefix[s.n - 2] : 0) < s.one))) {
            sh.sum.mass = 0;
            TQ1_DO(kAbove);
            s.kept = s.any ? min(s.kept, sh.sum.mass) : sh.sum.mass;
          } else if (!(s.any && s.weight_at >= s.one)) {  // else the last token kept so far weighs enough, so all do
            s.many = true;
            // A list whose last token weighs nearly min_p mostly holds the pick: then
            // what is kept is added up, and the list asked (512 rows of 32000 with a
            // min_p of 0.05 30 us, by bins 50; with 0.001 by bins 94, else 118).
            s.by_bin = s.whole && s.n > 0 && (s.in_list - (s.n > 1 ? sh.prefix[s.n - 2] : 0)) / 3 < s.one ? -1 : bin_of_weight(f.min_p);
            if (s.by_bin >= 0) {
              // What is kept ends in this bin: as where it ends by mass.
              s.whole = false;
              if (s.window != 0) {
                TQ1_DO(s.first ? ask(kMerge, 0, 0, 0) : ask(kMasses | kCounts | kMerge, 0, kCuts - 1, 0));
                s.window = 0;
                s.first = false;
              }
              s.mass0 = s.count0 = 0;
              s.pair = false;
              TQ1_DO(kSearch);
              s.b1 = s.by_bin;
              s.by_bin = -1;
              s.before = s.mass_before[0];
              s.tokens = 0;
              s.targets[0] = pick_of(f.u, max(u64{1}, s.before));
              s.targets[1] = pick_of(f.u, max(u64{1}, s.before + mass_of_bin(sh, s.b1)));
              s.pair = true;
              s.bin[0] = s.bin[1] = 0;
              TQ1_DO(kSearch);
              if (fit(sh, s.bin[0], s.bin[1], s.b1)) {
                TQ1_DO(ask(kGather, s.bin[0], s.bin[1] - s.bin[0], 0, 0, 0, 0, s.b1));
                if (sh.sum.n <= kList) {
                  s.kept = s.before;  // if nothing of the bin weighs enough
                  take_pair(sh, s);
                  s.n = static_cast<int>(sh.sum.n);
                  s.many = false;
                  TQ1_DO(kOrder);
                  sh.sum.mass = 0;
                  TQ1_DO(kAbove);
                  s.kept = max(s.kept, sh.sum.mass);
                }
              }
            }
            if (s.many) {
              s.picks = 0;
              TQ1_DO(ask(kWeigh, 0, 0, 0, s.one));
              s.kept = s.any ? min(s.kept, sh.sum.mass) : sh.sum.mass;
            }
          }
        }
        s.by_mass = s.question > 0;
        if (s.question == 2) s.token = -1;
        if (s.question == 0) s.target = static_cast<u64>(f.top_k);
        else if (s.question == 1) s.target = f.top_p > 0.0f ? max(u64{1}, part_of(s.kept, f.top_p, true)) : 1;
        else s.target = pick_of(f.u, s.kept);
        s.found = false;  // without the list
        if (s.whole && !s.ordered) {
          // What is asked of a list that holds the first top_k, or all, is answered there.
          s.leave = !s.gone && (s.complete || (s.question == 0 && f.top_k <= s.n));
          s.gone |= s.leave;
          TQ1_DO(kOrder);
          s.ordered = true;
        }
        if (!(s.question == 2 && s.picks && s.target > s.before && s.target <= sh.prefix[s.picks - 1]) &&
            !(s.whole && (s.complete || s.target <= (s.by_mass ? s.in_list : static_cast<u64>(s.n))))) {
          s.whole = s.by_key = false;
          s.picks = 0;
          s.split = 0xffffffffu;
          s.mass0 = s.count0 = s.tokens = s.gap = 0;
          s.i = s.shift = 0;
          for (;;) {  // windows of bins; then, of a bin of too many tokens, ranges of keys: every turn cuts them to a 1024th or less
            if (s.by_key) {
              s.shift = 0;
              while (((s.khi - s.klo) >> s.shift) >= kCuts) ++s.shift;
              TQ1_DO(ask(kByKey | kMasses | kCounts | kMerge, s.klo, s.khi - s.klo, s.shift));
              s.window = -1;
            } else if (s.window != s.i) {
              TQ1_DO(s.i == 0 && s.first ? ask(kMerge, 0, 0, 0) : ask(kMasses | kCounts | kMerge, s.i * kCuts, kCuts - 1, 0));
              s.window = s.i;
            }
            s.first = false;  // merged, or overwritten
            s.pair = false;
            s.targets[0] = s.target;
            s.bin[0] = 0;
            TQ1_DO(kSearch);
            if (!s.by_key && (s.by_mass ? s.mass0 + s.all_mass : s.count0 + s.all_count) < s.target) {
              s.mass0 += s.all_mass;
              s.count0 += s.all_count;
              if (++s.i < kWindows) continue;
              s.mass_at = s.mass0;  // fewer tokens than top_k: all of them
              s.weight_at = 0;
              s.found = true;
              break;
            }
            s.before = s.mass_before[0];
            s.tokens = s.count_before[0];
            if (!s.by_key) {
              s.b1 = s.bin[0];
              if (s.i == 0 && !f.by_m && s.question == (f.by_p ? 1 : 0)) {
                // What is kept ends in this bin, so the bins are known, mostly one,
                // that the pick can be in: they are gathered with it.
                s.targets[0] = pick_of(f.u, s.before + 1);
                s.targets[1] = pick_of(f.u, s.before + mass_of_bin(sh, s.b1));
                s.pair = true;
                s.bin[0] = s.bin[1] = 0;
                TQ1_DO(kSearch);
                if (fit(sh, s.bin[0], s.bin[1], s.b1)) {
                  TQ1_DO(ask(kGather, s.bin[0], s.bin[1] - s.bin[0], 0, 0, 0, 0, s.b1));
                  if (sh.sum.n <= kList) {
                    take_pair(sh, s);
                    break;
                  }
                }
              }
              s.many = s.i == 0 && tokens_of_bin(sh, s.b1) > 1.1f * kList;  // too many to gather
              s.b1 += s.i * kCuts;
              if (!s.many) {
                TQ1_DO(ask(kGather, s.b1, 0, 0));
                if (sh.sum.n <= kList) break;
              }
              TQ1_DO(ask(kRange, s.b1, 0, 0));
              s.klo = sh.sum.kmin;
              s.khi = sh.sum.kmax;
              s.by_key = true;
            } else {
              s.klo += min(static_cast<uint32_t>(s.bin[0]), (s.khi - s.klo) >> s.shift) << s.shift;
              s.khi = min(s.khi, s.klo + ((1u << s.shift) - 1u));
              if (sh.count[s.bin[0]] <= kList) {
                TQ1_DO(ask(kByKey | kGather, s.klo, s.khi - s.klo, 0));
                if (sh.sum.n > kList) {  // more than were counted
                  s.token = -1;
                  s.leave = !s.gone;
                  return kEnd;
                }
                break;
              }
              if (s.klo == s.khi) {  // more tokens than the list holds share one logit: they are counted off by index
                s.one = weight_of(sh.pow, sh.scale, logit_of(s.klo));
                s.nth = s.by_mass ? (s.target > s.before && s.one ? (s.target - s.before + s.one - 1) / s.one : 1) : s.target - s.tokens;
                s.nth = max(u64{1}, min(s.nth, static_cast<u64>(sh.count[s.bin[0]])));
                s.mass_at = s.before + s.nth * s.one;
                s.weight_at = s.one;
                if (s.question == 2) {
                  TQ1_DO(ask(kByKey | kTally, s.klo, 0, 0));
                  for (s.b0 = 0; static_cast<int>(s.b0) < sh.row.ranks - 1 && s.nth > sh.sum.tally[s.b0]; ++s.b0) s.nth -= sh.sum.tally[s.b0];
                  TQ1_DO(ask(kByKey | kFind, s.klo, 0, 0, 0, s.b0, static_cast<int>(s.nth)));
                  s.token = sh.sum.found - 1;
                }
                s.found = true;
                break;
              }
            }
            s.mass0 = s.before;
            s.count0 = s.tokens;
          }
          if (!s.found) {
            s.n = static_cast<int>(min(sh.sum.n, static_cast<unsigned>(kList)));
            s.skipped = s.tokens;
            TQ1_DO(kOrder);
          }
        } else if (s.question == 2) {
          s.leave = !s.gone;
          s.gone = true;
        }
        if (!s.found) {
          s.last = s.question == 2 && s.gone;
          TQ1_DO(kLookUp);
        }
        if (s.question < 2) s.kept = s.mass_at;
        s.any = true;
      }
  }
  s.leave = !s.gone;
  return kEnd;
}
#undef TQ1_DO

template <typename T, int N>
__global__ void __launch_bounds__(N, 1024 / N) sample_kernel(const SampleArgs a, int ranks, int one_wave, unsigned* status) {
  constexpr int kWarps = N / 32, kUnused = sizeof(T) == 2 ? (std::is_same<T, __half>::value ? 13 : 16) : 0;
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / ranks;
  const int rank = static_cast<int>(blockIdx.x) - static_cast<int>(r) * ranks;
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
  if (tid < 256) sh.pow[tid] = kPowers.w[tid];
  if (tid == 0) {
    const char* p = static_cast<const char*>(a.logits) + r * a.ld * static_cast<int64_t>(sizeof(T));
    constexpr int kVec = 16 / sizeof(T);
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    const int groups = (a.v + off + kVec - 1) / kVec, per = (groups + ranks - 1) / ranks;
    const int j0 = min(groups, rank * per);
    sh.row = {p, a.v, off, j0, min(groups, j0 + per), rank, ranks, false};
    sh.sum.mass = 0;
    sh.sum.n = 0;
  }
  __syncthreads();
  pdl_wait();
  if (one_wave) pdl_launch_dependents();

  if (tid == 0) {
    Filters f;
    f.temperature = a.temperature ? __ldcg(a.temperature + r) : 1.0f;
    f.top_k = a.top_k ? __ldcg(a.top_k + r) : 0;
    f.top_p = a.top_p ? __ldcg(a.top_p + r) : 1.0f;
    f.min_p = a.min_p ? __ldcg(a.min_p + r) : 0.0f;
    f.u = __ldcg(a.u + r);
    f.greedy = !(f.temperature > 7.888609052210118e-31f) || f.top_k == 1;  // 2^-100
    f.by_k = f.top_k > 0 && f.top_k < a.v;
    f.by_p = f.top_p < 1.0f;
    f.by_m = f.min_p > 0.0f;
    sh.own = f;
  }

  // The largest logit and its first token.
  float best = -INFINITY;
  int at = INT_MAX;
  {
    const Row<T, N> row;
    int group = -1;
    auto larger = [&](const float (&one)[Row<T, N>::kVec], int g) {
      float m = one[0];  // NaN: the other one
#pragma unroll
      for (int c = 1; c < Row<T, N>::kVec; ++c) m = fmaxf(m, one[c]);
      if (m > best || (m == best && g < group)) {
        best = m;
        group = g;
      }
      return false;
    };
    float one[Row<T, N>::kVec];
    row.scan(larger, [&](int g) {
      row.unpack(row.load(g), one);
      larger(one, g);
    });
    if (group >= 0) {
      row.unpack(row.load(group), one);
#pragma unroll
      for (int c = Row<T, N>::kVec - 1; c >= 0; --c)
        if (one[c] == best) at = group * Row<T, N>::kVec - row.off + c;
    }
    best += 0.0f;  // -0 equals 0
  }
  // Threads with nothing but masked logits, be the mask a type's lowest value, do not count below.
  const bool live = best > -1e30f;
  const uint32_t mine_key = live ? key_of(best) : 0xffffffffu;
  uint32_t low = live ? mine_key : 0u;  // the smallest of the threads' largest, as a key
  auto better = [](float l, int i, float m, int j) { return l > m || (l == m && i < j); };
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float l = __shfl_xor_sync(0xffffffffu, best, o);
    const int i = __shfl_xor_sync(0xffffffffu, at, o);
    if (better(l, i, best, at)) {
      best = l;
      at = i;
    }
  }
  low = __reduce_max_sync(0xffffffffu, low);
  if (lane == 0) {
    sh.red[warp] = best;
    sh.red_at[warp] = at;
    sh.red_low[warp] = low;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    low = max(low, sh.red_low[i]);
    if (better(sh.red[i], sh.red_at[i], best, at)) {
      best = sh.red[i];
      at = sh.red_at[i];
    }
  }
  // A list to begin with: where `wanted` threads of the cluster have a logit
  // of at least x, so many tokens have one.  Each CTA finds an x for its share
  // of the threads; the smallest of them serves.  Of nearly as many as there are
  // threads x would be too low: the list too long.
  auto wanted_of = [&](const Filters& f) {
    return ((f.by_k ? min(f.top_k, kMostWanted + 1) : a.v <= kShortRow ? max(kWanted, min(N / 2, a.v / 16)) : kWanted) + ranks - 1) / ranks;
  };
  auto lists_of = [&](const Filters& f) { return !f.greedy && (!f.by_k || f.top_k <= kMostWanted) && wanted_of(f) <= N / 8 * 7; };
  const int wanted = wanted_of(sh.own);
  float least = -INFINITY;  // fewer threads than wanted have any: all tokens
  if (lists_of(sh.own) && __syncthreads_count(mine_key != 0xffffffffu) >= wanted) {
    // Halved by value, and by key every other time: a few logits far from the
    // rest, or many about zero, hold up one of the two.
    uint32_t hi = key_of(best);
#pragma unroll 1
    for (int turn = 0; turn < 16 && low > hi; ++turn) {
      uint32_t mid = hi + (low - hi) / 2;
      if (!(turn & 1)) mid = max(hi, min(low - 1, key_of(0.5f * logit_of(hi) + 0.5f * logit_of(low) + 0.0f)));
      const int n = __syncthreads_count(mine_key <= mid);
      if (n < wanted) {
        hi = mid + 1;
        continue;
      }
      low = mid;
      if (n <= wanted + min(wanted / 2, (N - wanted) / 8)) break;
    }
    least = logit_of(low);
  }
  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // and so do the others
  if (tid < ranks) {
    Shared& to = ranks == 1 ? sh : shared_of(tid);
    to.best[rank] = best;
    to.best_at[rank] = at;
    to.least[rank] = least;
    if (rank == 0) to.filters = sh.own;
  }
  sync_row(ranks);
  const Filters& filters = sh.filters;
  for (int i = 0; i < ranks; ++i) {
    least = fminf(least, sh.least[i]);
    if (better(sh.best[i], sh.best_at[i], best, at)) {
      best = sh.best[i];
      at = sh.best_at[i];
    }
  }
  if (filters.greedy || best == -INFINITY) {
    if (rank == 0 && tid == 0) {
      a.ids[r] = best == -INFINITY ? -1 : at;
      if (a.probs) a.probs[r] = best == -INFINITY ? 0.0f : 1.0f;
    }
    return;
  }

  // The list, and the masses where that of everything will be asked for.
  const bool lists = lists_of(filters), all = !filters.by_k && (filters.by_p || !filters.by_m);
  if (tid == 0) {
    const bool top = best == INFINITY;
    // 2 log2(e) / T: the quotient, and what the rounding of it left over.
    const float log2e = 2.88539004325866699219f, log2e_lo = 3.85192598e-8f;  // twice, for the halves
    Scale s;
    s.max = top ? 0.0f : 0.5f * best;
    s.c = __fdiv_rn(log2e, filters.temperature);
    s.c_lo = __fdiv_rn(fmaf(-s.c, filters.temperature, log2e) + log2e_lo, filters.temperature);
    if (filters.temperature == INFINITY) s.c = s.c_lo = 0.0f;  // all alike
    sh.scale = s;
    sh.row.top = top;
    Command c = {(all ? kWeigh | kMasses : 0) | (lists ? kTop : 0), 0, all ? kCuts - 1u : 0u, kNoBin, 0, least, {0.0f, 0.0f}, {INFINITY, INFINITY}, 0, 0, 0};
    if (!top) middle_of(least, best, c.mid[0], c.half[0]);
    sh.cmd = c;
  } else if (tid == 32) {  // a warp that has nothing else to do
    State& s = sh.state;
    s.at = 0;
    s.ordered = false;
    s.before = s.skipped = s.gap = 0;
    s.picks = 0;
    s.split = 0xffffffffu;
    s.by_bin = -1;
    s.mass_at = s.weight_at = 0;
    s.token = 0;
    s.any = s.first = all;
    s.gone = ranks == 1;
    s.window = -1;
  }
  __syncthreads();
  if (all || lists) pass<T, N>();
  if (rank != 0) {  // do what the leader asks for
    for (;;) {
      sync_row(ranks);
      if (sh.cmd.flags == kDone) return;
      pass<T, N>();
    }
  }

  if (tid == 0) {
    State& s = sh.state;
    s.n = static_cast<int>(min(sh.sum.n, static_cast<unsigned>(kList)));
    s.whole = lists && sh.sum.n <= kList;
    s.complete = s.whole && least == -INFINITY;
    s.kept = sh.sum.mass;
  }
#pragma unroll 1
  for (;;) {
    if (tid == 0) sh.state.act = decide();
    __syncthreads();
    // Read here: behind the next barrier thread 0 may be deciding anew.
    const int act = sh.state.act;
    const bool leave = sh.state.leave, last = sh.state.last;
    if (leave) dismiss(ranks);
    if (act == kPass) {
      if (tid < ranks) (ranks > 1 ? shared_of(tid) : sh).cmd = sh.next;
      sync_row(ranks);
      pass<T, N>();
    } else if (act == kOrder) {
      order<N>(kUnused);
    } else if (act == kSearch) {
      search<N>();
    } else if (act == kEnd) {
      break;
    } else {
      const State& s = sh.state;
      for (int i = tid; i < s.n; i += N) {
        if (act == kAbove) {
          const u64 upto = sh.prefix[i], below = i ? sh.prefix[i - 1] + (i == s.picks ? s.gap : 0) : s.before;
          if (upto - below >= s.one) atomicMax(&sh.sum.mass, upto);
          continue;
        }
        const int place = sh.place[i];
        const u64 upto = sh.prefix[place], below = place ? sh.prefix[place - 1] : s.before;
        if (s.by_mass ? (below < s.target && upto >= s.target)
                      : (s.skipped + place + 1 == s.target || (s.complete && place == s.n - 1 && s.target > static_cast<u64>(s.n)))) {
          sh.state.mass_at = upto;
          sh.state.weight_at = upto - below;
          sh.state.token = static_cast<int>(static_cast<uint32_t>(sh.list[i]));
        }
      }
      __syncthreads();
      if (last) break;
    }
  }
  if (tid == 0) {
    a.ids[r] = sh.state.token;
    if (a.probs) a.probs[r] = sh.state.token < 0 ? 0.0f : ratio_of(sh.state.weight_at, sh.state.kept);
    if (sh.state.token < 0) raise_status(status, kStatusBadId);
  }
}

constexpr int kOnePerSm = 120 * 1024;  // shared memory of which an SM holds one CTA's
static_assert(sizeof(Shared) <= 76 * 1024 && sizeof(Shared) <= kOnePerSm, "two CTAs an SM");

template <typename T, int N>
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};

  Launch(int64_t ctas, int ranks, size_t smem, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(N);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Launch(const Launch&) = delete;
};

// Allows the kernel its shared memory on the current device, once a device
// (racing threads do it twice: idempotent).
template <typename T, int N>
int configure(int dev) {
  static std::atomic<bool> done[64];
  if (!done[dev].load(std::memory_order_acquire)) {
    if (!cuda_ok(cudaFuncSetAttribute(sample_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOnePerSm))) return TQ1_ERR_CUDA;
    done[dev].store(true, std::memory_order_release);
  }
  return TQ1_OK;
}

// How many clusters of so many CTAs of 512 threads the device holds at once,
// one CTA or two an SM: fewer than SMs / ranks, since a cluster's SMs are of
// one group (a GB300's 152 SMs hold 36 clusters of four, 15 of eight).
template <typename T>
int64_t clusters(int dev, int ranks, bool two) {
  static std::atomic<int> known[64][2][kMaxCluster + 1];  // plus one
  std::atomic<int>& k = known[dev][two][ranks];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    Launch<T, 512> l(ranks, ranks, two ? sizeof(Shared) : static_cast<size_t>(kOnePerSm), nullptr);
    l.cfg.numAttrs = 1;
    if (!cuda_ok(cudaOccupancyMaxActiveClusters(&n, sample_kernel<T, 512>, &l.cfg))) n = 0;
    ++n;
    k.store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

template <typename T, int N>
int launch(const SampleArgs& a, int64_t t, int ranks, int one_wave, unsigned* status, cudaStream_t s) {
  Launch<T, N> l(t * ranks, ranks, sizeof(Shared), s);
  return cuda_ok(cudaLaunchKernelEx(&l.cfg, sample_kernel<T, N>, a, ranks, one_wave, status)) ? TQ1_OK : TQ1_ERR_CUDA;
}

// Rows beyond two an SM: a CTA of 256 threads each (512 rows of 32000 take 0.82
// of the time with 512 threads).  Else CTAs of 512 (with 1024 one row of 131072
// takes 1.3 times as long), and as many a row as find an SM of their own (24 rows
// of 200003, five a row: 0.83 of the time with eight; 100 rows of 32000, one: 0.80 of
// the time with two), 2048 tokens each at the least (a row of 4000, one: 0.92 of the
// time with two).  Long rows of which that leaves one CTA or two have as many as fit
// two an SM (50 rows of 200003, five: 0.84 of the time with two; of 50000 1.07).
constexpr int kLongRow = 98304;

template <typename T>
int launch_type(const SampleArgs& a, int64_t t, unsigned* status, cudaStream_t s) {
  const int dev = device_info().device;
  if (dev < 0 || dev >= 64) return TQ1_ERR_CUDA;
  if (configure<T, 512>(dev) != TQ1_OK || configure<T, 256>(dev) != TQ1_OK) return TQ1_ERR_CUDA;
  const int64_t sms = std::max(1, device_info().num_sms);
  if (t > 2 * sms) return launch<T, 256>(a, t, 1, t <= 4 * sms, status, s);
  auto most = [&](bool two) {
    int ranks = kMaxCluster;
    while (ranks > 1 && (a.v < ranks * 2048 || clusters<T>(dev, ranks, two) < t)) --ranks;
    return ranks;
  };
  int ranks = most(false);
  if (ranks <= 2 && a.v >= kLongRow) ranks = most(true);
  return launch<T, 512>(a, t, ranks, 1, status, s);
}

}  // namespace

int launch_sample(const SampleArgs& a, int64_t t, unsigned* status, cudaStream_t s) {
  switch (a.type) {
    case kF16: return launch_type<__half>(a, t, status, s);
    case kBf16: return launch_type<__nv_bfloat16>(a, t, status, s);
    default: return launch_type<float>(a, t, status, s);
  }
}

}  // namespace tq1
