// moe_layer.cu -- a mixture-of-experts layer for a few tokens:
//   ids, p = the top_k largest of a token's logits, their softmax weights
//   h_s    = Q8_1(silu(G x) * (U x))
//   out    = res + sum_s p_s D h_s
// with G, U [f][k] and D [k][f] of expert ids_s, ternary, on the decode
// kernels' packed digits and masked dp4a (exact integer partials, fp32 scales).
//
// Selection is a warp's work: a lane keeps a 32nd of the logits, each place of
// the order is one maximum over the lanes.
//
// Few pairs (token, slot): two kernels.  In the first a CTA takes one pair and
// 32 rows of h, so it has both products of its rows and whole Q8_1 blocks of
// h; it selects the expert itself, while its other warps lay out the
// activations.  In the second a CTA takes one token and a range of output
// rows, and all of the token's slots, so the weighted sum is formed where the
// products are, in the order of the slots; its weights are fetched and
// expanded while the first kernel still runs.
//
// More pairs: several tokens share an expert, whose rows are then expanded
// once for up to six of them.  A kernel selects, one warp a token; the two
// product kernels walk tasks (expert, up to six of its pairs, a range of
// rows) that every CTA finds from the ids in shared memory; a last one adds up.
//
// One token waits for the chain of selection, weights and h (8 of 128 experts of
// 768 x 2048 in 10.2 us).  Large experts and batches expand and multiply, but fill no
// pipe: issue slots are 48 to 60% used, that of integer products 41 to 55%; the
// rest are waits for staged weights, turns that end unevenly, and selection and sum in
// kernels of their own.  7 tokens of two of 8 experts of 2816 x 4096 42 us, 32 tokens of
// 8 of 128 89 us.  From some 16 pairs an expert on a pair costs the same however many
// there are (512 tokens of 8 of 128 0.82 ms, 47 TOP/s): there are no tensor cores here.
//
// Units are (row, 256-block): a lane expands one block and multiplies it.  Four
// neighbouring lanes take the same block of four rows, so that their readings of
// the activations' record coincide: with eight different records a warp, 16-byte
// reads take 2.3 cycles when equal ones stand side by side, 4.0 when every
// eighth lane's are equal, and these kernels wait for little else as long.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/tq1.h"
#include "kv.cuh"
#include "packed.cuh"
#include "step_internal.h"
#include "tq1_device.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

using namespace packed;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHRows = 32;  // rows of h a CTA forms at a time: one Q8_1 block
constexpr int kMaxTop = 32;
// Pairs that share an expansion: 32 tokens of 8 of 128 experts of 768 x 2048
// take 95.6, 88.7 and 90.1 us with up to four, six and eight.  TQ2_0, which
// has little to expand, 76.7, 76.9 and 76.4, 12 tokens of two of 8 experts of
// 2816 x 4096 49, 55 and 54.
template <int FMT>
constexpr int kChunk = FMT == kFmtTq2 ? 4 : 6;
constexpr size_t kMaxSmem = 200 * 1024;
constexpr size_t kHalfSmem = 112 * 1024;  // two CTAs an SM
constexpr size_t kThirdSmem = 74 * 1024;

// ------------------------------------------------------------- selection --
// Larger logits have larger keys; NaN and -inf, which are never selected, 0.
__device__ __forceinline__ uint32_t select_key(float l) {
  if (!(l > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 equals 0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float selected_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

constexpr int kMaxExperts = 1024;

// By one warp: lane s gets the expert in place s of the token's order and its
// weight (-1 and 0 where there is none), for s < rounds.  Weights are formed
// only where all places are (rounds == top_k).  A lane keeps every 32nd logit
// and knows the largest of them, which only the lane that gives one away has
// to find again: among four registers, or (kMany) in shared memory of the
// warp's own, `keys`.
template <bool kMany>
__device__ __forceinline__ void route_lanes(const MoeLayerArgs& a, int64_t token, int rounds, uint32_t* keys, int& expert, float& weight) {
  const int lane = threadIdx.x & 31, n = a.n_experts;
  uint32_t own[4] = {0, 0, 0, 0}, best = 0;
  int at = 0;
  auto each = [&](auto&& f) {
    if constexpr (kMany) {
#pragma unroll 4
      for (int e = lane; e < n; e += 32) f(e, keys[e]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f(lane + 32 * i, own[i]);
    }
  };
  auto find = [&]() {
    best = 0;
    each([&](int e, uint32_t& k) {
      if (k > best) {
        best = k;
        at = e;
      }
    });
  };
  // From L2: kernels that begin early read them while others end.
  each([&](int e, uint32_t& k) { k = e < n ? select_key(__ldcg(a.logits + token * n + e)) : 0; });
  find();
  expert = -1;
  weight = 0.0f;
  const uint32_t top = __reduce_max_sync(0xffffffffu, best);
  const bool weigh = rounds == a.top_k;
  auto part = [&](uint32_t k) {  // exp(l - largest); where the largest is +inf, only its like count
    if (k == 0) return 0.0f;
    return top == select_key(INFINITY) ? (k == top ? 1.0f : 0.0f) : expf(selected_logit(k) - selected_logit(top));
  };
  float sum = 0.0f;
  if (weigh && !a.renormalize) each([&](int, uint32_t& k) { sum += part(k); });
  uint32_t mine = 0;
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    if (most == 0) break;  // nothing is left
    const int e = __reduce_min_sync(0xffffffffu, best == most ? at : 0x7fffffff);
    if (lane == r) {
      expert = e;
      mine = most;
    }
    if (!kMany || (e & 31) == lane) {
      each([&](int i, uint32_t& k) {
        if (i == e) k = 0;
      });
      find();
    }
  }
  if (!weigh) return;
  const float own_part = part(mine);
  if (a.renormalize) sum = own_part;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (mine) weight = a.scale * __fdiv_rn(own_part, sum);
}
__device__ __forceinline__ void route(const MoeLayerArgs& a, int64_t token, int rounds, uint32_t* keys, int& expert, float& weight) {
  if (a.n_experts <= 128) route_lanes<false>(a, token, rounds, keys, expert, weight);
  else route_lanes<true>(a, token, rounds, keys, expert, weight);
}

// ---------------------------------------------------------------- pieces --
// Requests `bytes` weight bytes from src (16-byte pieces that cover them; the
// last bytes of the matrices, past the last whole piece, with plain loads)
// into dst, which has room for 15 bytes more on either side.  One thread.
__device__ __forceinline__ void request(uint8_t* dst, const uint8_t* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  const uint32_t delta = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
  const uint32_t tot = delta + bytes, main = tot & ~15u;
  const uint8_t* from = src - delta;
  for (uint32_t i = main; i < tot; ++i) dst[i] = from[i];
  mbar_arrive_expect_tx(bar, main);
  if (main) bulk_g2s(dst, from, main, bar, policy);
}
// Shared memory of a region of so many weight bytes: the alignment before,
// the expansion's reads behind.
__host__ __device__ __forceinline__ uint32_t region(uint32_t bytes) { return (bytes + 15u + 16u + 15u) & ~15u; }
__device__ __forceinline__ uint32_t low4(const uint8_t* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u); }

// Unit u of rows of nb blocks (their number a multiple of four).
struct Unit {
  int row, block;
};
__device__ __forceinline__ Unit unit_of(int u, int nb) {
  const int four = u / (4 * nb), in = u - four * 4 * nb;
  return {4 * four + (in & 3), in >> 2};
}
// Partials of a row are an odd number of words apart from the next row's, so
// that lanes that add up a row each meet in no bank.
__host__ __device__ __forceinline__ int pitch_of(int nb) { return nb | 1; }

// d_w sum_j d_a[j] I_j of one packed block against two records: the masks of
// its slots are formed once for both.
__device__ __forceinline__ void packed_dot_two(const Packed& P, const uint32_t* r, const uint32_t* s, float& x, float& y) {
  int I[8], J[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int4 a = *reinterpret_cast<const int4*>(r + 72 + 4 * h), b = *reinterpret_cast<const int4*>(s + 72 + 4 * h);
    I[4 * h] = a.x; I[4 * h + 1] = a.y; I[4 * h + 2] = a.z; I[4 * h + 3] = a.w;
    J[4 * h] = b.x; J[4 * h + 1] = b.y; J[4 * h + 2] = b.z; J[4 * h + 3] = b.w;
  }
#pragma unroll
  for (int w = 0; w < 8; ++w) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 a = *reinterpret_cast<const uint4*>(r + 8 * w + 4 * h), b = *reinterpret_cast<const uint4*>(s + 8 * w + 4 * h);
      const uint32_t q = h ? P.b[w] : P.a[w];
      const uint32_t m0 = q & 0x03030303u, m1 = q & 0x0C0C0C0Cu, m2 = q & 0x30303030u, m3 = q & 0xC0C0C0C0u;
      I[4 * h] = dp4a_us(m0, a.x, I[4 * h]);
      J[4 * h] = dp4a_us(m0, b.x, J[4 * h]);
      I[4 * h + 1] = dp4a_us(m1, a.y, I[4 * h + 1]);
      J[4 * h + 1] = dp4a_us(m1, b.y, J[4 * h + 1]);
      I[4 * h + 2] = dp4a_us(m2, a.z, I[4 * h + 2]);
      J[4 * h + 2] = dp4a_us(m2, b.z, J[4 * h + 2]);
      I[4 * h + 3] = dp4a_us(m3, a.w, I[4 * h + 3]);
      J[4 * h + 3] = dp4a_us(m3, b.w, J[4 * h + 3]);
    }
  }
  x = packed_scale(I, r, P.dw);
  y = packed_scale(J, s, P.dw);
}
// The same block against `pairs` records, rstride words apart; to[c * tstride].
__device__ __forceinline__ void packed_dots(const Packed& P, const uint32_t* rec, int rstride, int pairs, float* to, int tstride) {
  int c = 0;
#pragma unroll 1
  for (; c + 2 <= pairs; c += 2, rec += 2 * rstride, to += 2 * tstride) packed_dot_two(P, rec, rec + rstride, to[0], to[tstride]);
  if (c < pairs) *to = packed_dot(P, rec);
}

// The products of a run of rows (a multiple of four, contiguous, nb blocks
// each) with `pairs` records' sets, to part[c * pstride + row * pitch_of(nb) + block];
// and of a second run of as many rows at off2 (if any), its partials part2 words on.
// All places are bytes of shared memory.  Not inlined: what its callers keep
// beside would not fit the registers that three CTAs an SM leave a thread.
template <int FMT>
__device__ __noinline__ void rows_dots(uint32_t off, uint32_t off2, int part2, int nb, int rows, uint32_t recs_at, int pairs,
                                       uint32_t part_at, int pstride) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t* recs = reinterpret_cast<const uint32_t*>(smem + recs_at);
  float* part = reinterpret_cast<float*>(smem + part_at);
  const int units = rows * nb, all = off2 ? 2 * units : units;
#pragma unroll 1
  for (int u = threadIdx.x; u < all; u += kThreads) {
    const bool second = u >= units;
    const Unit x = unit_of(second ? u - units : u, nb);
    Packed P;
    unit_pack<FMT>(smem, (second ? off2 : off) + static_cast<uint32_t>(x.row * nb + x.block) * fmt_block_bytes<FMT>(), P);
    packed_dots(P, recs + x.block * kPRec, nb * kPRec, pairs, part + (second ? part2 : 0) + x.row * pitch_of(nb) + x.block, pstride);
  }
}

// silu(g) u of 32 rows, lane's row, as a Q8_1 block: the quantiser's operations.
__device__ __forceinline__ void store_h(float g, float u, uint8_t* block) {
  const int lane = threadIdx.x & 31;
  const float h = __fdiv_rn(g, 1.0f + expf(-g)) * u;
  float m = fabsf(h);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = __fdiv_rn(m, 127.0f);
  int q = 0;
  if (d != 0.0f) q = static_cast<int>(fminf(fmaxf(roundf(__fdiv_rn(h, d)), -127.0f), 127.0f));
  const int sum = __reduce_add_sync(0xffffffffu, q);
  const uint32_t qb = static_cast<uint32_t>(q) & 0xFFu;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, qb, ((lane & 7) << 2) + i) << (8 * i);
  uint32_t* o = reinterpret_cast<uint32_t*>(block);
  if (lane < 8) o[1 + lane] = word;
  if (lane == 0) {
    const uint32_t d16 = __half_as_ushort(__float2half_rn(d));
    const uint32_t s16 = __half_as_ushort(__float2half_rn(__fmul_rn(d, static_cast<float>(sum))));
    o[0] = d16 | (s16 << 16);
  }
}

__device__ __forceinline__ void store_out(const MoeLayerArgs& a, int64_t at, float v) {
  if (a.res) v += a.res[at];
  if (a.out_type == kF32) static_cast<float*>(a.out)[at] = v;
  else if (a.out_type == kF16) static_cast<__half*>(a.out)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

// --------------------------------------------------------------- few pairs --
struct UpLayout {
  uint32_t slab, recs, part, total;
};
__host__ __device__ __forceinline__ UpLayout up_layout(int nb, int block_bytes, int pairs) {
  UpLayout l;
  l.slab = 2 * region(kHRows * nb * block_bytes);
  l.recs = l.slab;
  l.part = l.recs + pairs * nb * kPRec * 4;
  l.total = l.part + pairs * 2 * kHRows * pitch_of(nb) * 4;
  return l;
}

template <int FMT, int kUpThreads>
__global__ void __launch_bounds__(kUpThreads, 1024 / kUpThreads) moe_up_kernel(const MoeLayerArgs a, uint8_t* h8, unsigned* status) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int s_expert;
  __shared__ uint32_t s_keys[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = a.k / kQK, parts = a.f / kHRows;
  const int pair = static_cast<int>(blockIdx.x) / parts, part0 = static_cast<int>(blockIdx.x) - pair * parts;
  const int token = pair / a.top_k, slot = pair - token * a.top_k;
  const UpLayout l = up_layout(nb, kBB, 1);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + l.recs);
  float* part = reinterpret_cast<float*>(smem + l.part);
  const uint32_t rowbytes = static_cast<uint32_t>(nb) * kBB, bytes = kHRows * rowbytes;
  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  pdl_wait();
  // The second kernel reads the logits before this one has ended: it may begin
  // once every CTA here has seen the end of what wrote them.
  pdl_launch_dependents();
  if (warp == 0) {
    int expert;
    float weight;
    const bool tell = part0 == 0 && slot == 0 && (a.ids || a.weights);
    route(a, token, tell ? a.top_k : slot + 1, s_keys, expert, weight);
    const int e = __shfl_sync(0xffffffffu, expert, slot);
    if (lane == 0) s_expert = e;
    if (e >= 0 && lane < 2) {
      const int64_t at = (static_cast<int64_t>(e) * a.f + part0 * kHRows) * rowbytes;
      request(smem + lane * region(bytes), (lane ? a.up : a.gate) + at, bytes, &bars[lane], l2_evict_first_policy());
    }
    if (tell && lane < a.top_k) {
      if (a.ids) a.ids[static_cast<int64_t>(token) * a.top_k + lane] = expert;
      if (a.weights) a.weights[static_cast<int64_t>(token) * a.top_k + lane] = weight;
    }
  } else {
    for (int i = tid - 32; i < nb * 8; i += kUpThreads - 32)
      fill_precord_chunk(a.q8 + (static_cast<int64_t>(token) * nb * 8 + i) * kQ8Bytes, recs + (i >> 3) * kPRec, i & 7);
  }
  __syncthreads();
  const int e = s_expert;
  if (e < 0) return;  // no copy was issued
  const int64_t at = (static_cast<int64_t>(e) * a.f + part0 * kHRows) * rowbytes;
  const int units = kHRows * nb, pitch = pitch_of(nb);
  bool ok = true;
#pragma unroll 1
  for (int u = tid; u < 2 * units; u += kUpThreads) {
    const int m = u >= units;
    const Unit x = unit_of(u - (m ? units : 0), nb);
    ok = mbar_wait(&bars[m], 0);
    if (!ok) break;
    Packed P;
    unit_pack<FMT>(smem, m * region(bytes) + low4((m ? a.up : a.gate) + at) + static_cast<uint32_t>(x.row * nb + x.block) * kBB, P);
    part[(m * kHRows + x.row) * pitch + x.block] = packed_dot(P, recs + x.block * kPRec);
  }
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      raise_status(status, kStatusTimeout);
      for (int m = 0; m < 2; ++m) (void)mbar_wait(&bars[m], 0);  // let copies land (bounded)
    }
    return;
  }
  if (warp == 0) {
    float g = 0.0f, u = 0.0f;
#pragma unroll 4
    for (int b = 0; b < nb; ++b) {
      g += part[lane * pitch + b];
      u += part[(kHRows + lane) * pitch + b];
    }
    store_h(g, u, h8 + (static_cast<int64_t>(pair) * parts + part0) * kQ8Bytes);
  }
}

struct DownLayout {
  uint32_t slab, recs, part, total;
};
__host__ __device__ __forceinline__ DownLayout down_layout(int nbf, int block_bytes, int rows, int slots) {
  DownLayout l;
  l.slab = slots * region(rows * nbf * block_bytes);
  l.recs = l.slab;
  l.part = l.recs + slots * nbf * kPRec * 4;
  l.total = l.part + slots * rows * pitch_of(nbf) * 4;
  return l;
}

// `slots` slots of the token at a time (all of them where they fit).
template <int FMT>
__global__ void __launch_bounds__(kThreads, 3) moe_down_kernel(const MoeLayerArgs a, const uint8_t* h8, int rows, int slots,
                                                            unsigned* status) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ int s_expert[kMaxTop];
  __shared__ float s_weight[kMaxTop];
  __shared__ float s_acc[64];
  __shared__ uint32_t s_keys[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nbf = a.f / kQK, ranges = (a.k + rows - 1) / rows;
  const int token = static_cast<int>(blockIdx.x) / ranges, r0 = (static_cast<int>(blockIdx.x) - token * ranges) * rows;
  const int n = min(rows, a.k - r0);
  const DownLayout l = down_layout(nbf, kBB, rows, slots);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + l.recs);
  float* part = reinterpret_cast<float*>(smem + l.part);
  const uint32_t rowbytes = static_cast<uint32_t>(nbf) * kBB, span = region(rows * rowbytes);
  const int units = n * nbf;
  pdl_launch_dependents();
  uint32_t phase = 0;
  for (int s0 = 0; s0 < a.top_k; s0 += slots) {
    const int ns = min(slots, a.top_k - s0);
    if (warp == 0) {
      if (s0 == 0) {
        if (lane == 0) {
          mbar_init(&bar, 32);
          fence_mbar_init();
        }
        // The logits were complete before the first kernel let this one begin.
        int expert;
        float weight;
        route(a, token, a.top_k, s_keys, expert, weight);
        s_expert[lane] = expert;
        s_weight[lane] = weight;
        __syncwarp();
      } else {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // behind the plain stores and reads of the slots before
      }
      const int e = lane < ns ? s_expert[s0 + lane] : -1;
      if (e >= 0)
        request(smem + lane * span, a.down + (static_cast<int64_t>(e) * a.k + r0) * rowbytes, n * rowbytes, &bar, l2_evict_first_policy());
      else
        mbar_arrive_expect_tx(&bar, 0);
    }
    __syncthreads();
    auto pack = [&](int u, Packed& P) {  // whether there is such a unit
      const int s = u / units;
      const int e = s_expert[s0 + s];
      if (e < 0) return false;
      const uint32_t off = s * span + low4(a.down + (static_cast<int64_t>(e) * a.k + r0) * rowbytes);
      const Unit x = unit_of(u - s * units, nbf);
      unit_pack<FMT>(smem, off + static_cast<uint32_t>(x.row * nbf + x.block) * kBB, P);
      return true;
    };
    bool ok = mbar_wait(&bar, phase);
    phase ^= 1;
    Packed first;  // a thread's first unit is expanded before the wait for h
    const bool mine = ok && tid < ns * units && pack(tid, first);
    if (s0 == 0) pdl_wait();  // h is complete
    for (int i = tid; i < ns * nbf * 8; i += kThreads) {
      const int s = i / (nbf * 8), c = i - s * nbf * 8;
      if (s_expert[s0 + s] >= 0)
        fill_precord_chunk(h8 + ((static_cast<int64_t>(token) * a.top_k + s0 + s) * nbf * 8 + c) * kQ8Bytes,
                           recs + (s * nbf + (c >> 3)) * kPRec, c & 7);
    }
    __syncthreads();
    if (ok) {
      auto dot = [&](int u, const Packed& P) {
        const int s = u / units;
        const Unit x = unit_of(u - s * units, nbf);
        part[(s * n + x.row) * pitch_of(nbf) + x.block] = packed_dot(P, recs + (s * nbf + x.block) * kPRec);
      };
      if (mine) dot(tid, first);
#pragma unroll 1
      for (int u = tid + kThreads; u < ns * units; u += kThreads) {
        Packed P;
        if (pack(u, P)) dot(u, P);
      }
    }
    if (__syncthreads_or(!ok)) {
      if (tid == 0) {
        raise_status(status, kStatusTimeout);
        (void)mbar_wait(&bar, phase ^ 1);  // let copies land (bounded)
      }
      return;
    }
    // Weighted sums of each (slot, row)'s blocks, then of the slots in order.
    float* sums = reinterpret_cast<float*>(recs);  // the records are done with
    for (int i = tid; i < ns * n; i += kThreads) {
      const int s = i / n;
      float y = 0.0f;
      if (s_expert[s0 + s] >= 0)
        for (int b = 0; b < nbf; ++b) y += part[i * pitch_of(nbf) + b];
      sums[i] = s_weight[s0 + s] * y;
    }
    __syncthreads();
    for (int r = tid; r < n; r += kThreads) {
      float v = s0 ? s_acc[r] : 0.0f;
      for (int s = 0; s < ns; ++s) v += sums[s * n + r];
      if (s0 + slots < a.top_k) s_acc[r] = v;
      else store_out(a, static_cast<int64_t>(token) * a.k + r0 + r, v);
    }
    if (s0 + slots < a.top_k) __syncthreads();
  }
}

// -------------------------------------------------------------- more pairs --
// One warp a token: ids and weights into the workspace, and to the caller.
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const MoeLayerArgs a, int32_t* ids, float* weights) {
  __shared__ uint32_t s_keys[kWarps][kMaxExperts];
  const int lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (token >= a.t) return;
  int expert;
  float weight;
  route(a, token, a.top_k, s_keys[threadIdx.x >> 5], expert, weight);
  if (lane < a.top_k) {
    const int64_t at = token * a.top_k + lane;
    ids[at] = expert;
    weights[at] = weight;
    if (a.ids) a.ids[at] = expert;
    if (a.weights) a.weights[at] = weight;
  }
}

// The pairs by expert: pairs of expert e at plist[first[e]] .. (in order),
// its chunks from chunk[e] on.
struct Table {
  int *first, *chunk, *plist;
};
__host__ __device__ __forceinline__ uint32_t table_bytes(int n_experts, int pairs) {
  return static_cast<uint32_t>(2 * (n_experts + 1) + n_experts + pairs) * 4u;
}
// By all threads; returns the number of chunks of up to `most` pairs.
__device__ __forceinline__ int build_table(uint8_t* smem, const int32_t* ids, int n, int pairs, int most, Table& t) {
  const int tid = threadIdx.x, lane = tid & 31;
  t.first = reinterpret_cast<int*>(smem);
  t.chunk = t.first + n + 1;
  int* cursor = t.chunk + n + 1;
  t.plist = cursor + n;
  for (int e = tid; e < n; e += kThreads) cursor[e] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += kThreads) {
    const int e = __ldcg(ids + p);
    if (e >= 0) atomicAdd(&cursor[e], 1);
  }
  __syncthreads();
  if (tid < 32) {
    int before = 0, chunks = 0;
    for (int base = 0; base < n; base += 32) {
      const int e = base + lane, c = e < n ? cursor[e] : 0, q = (c + most - 1) / most;
      int x = c, y = q;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
          x += u;
          y += v;
        }
      }
      if (e < n) {
        t.first[e] = cursor[e] = before + x - c;
        t.chunk[e] = chunks + y - q;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
      chunks += __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) {
      t.first[n] = before;
      t.chunk[n] = chunks;
    }
    __syncwarp();
    for (int base = 0; base < pairs; base += 32) {  // in the order of the pairs
      const int p = base + lane;
      const int e = p < pairs ? __ldcg(ids + p) : -1;
      const uint32_t peers = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(peers & ((1u << lane) - 1u));
      if (e >= 0) t.plist[cursor[e] + rank] = p;
      __syncwarp();
      if (e >= 0 && rank == 0) cursor[e] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  return t.chunk[n];
}

// A task's expert and pairs.
struct Task {
  int expert, first, pairs;
};
__device__ __forceinline__ Task find_task(const Table& t, int n, int chunk) {
  int lo = 0, hi = n - 1;  // the last expert whose chunks begin at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  // An expert's chunks are even.
  const int pairs = t.first[lo + 1] - t.first[lo], chunks = t.chunk[lo + 1] - t.chunk[lo], each = (pairs + chunks - 1) / chunks;
  Task x;
  x.expert = lo;
  x.first = t.first[lo] + (chunk - t.chunk[lo]) * each;
  x.pairs = min(each, t.first[lo + 1] - x.first);
  return x;
}

// The parity of a barrier that completes once a turn.
__device__ __forceinline__ uint32_t slot_phase(int turn) { return static_cast<uint32_t>(turn) & 1u; }

struct UpTaskLayout {
  uint32_t recs, part, total;
};
__host__ __device__ __forceinline__ UpTaskLayout up_task_layout(int nb, int block_bytes, int pairs, int stage_rows) {
  UpTaskLayout l;
  l.recs = 4 * region(stage_rows * nb * block_bytes);
  l.part = l.recs + pairs * nb * kPRec * 4;
  l.total = l.part + pairs * 2 * kHRows * pitch_of(nb) * 4;
  return l;
}

// What a task is, in shared memory: the next one's is found while this one's
// products are formed.
struct TaskInfo {
  int first, pairs, range;
  const uint8_t* src[2];  // first product: its rows of gate and up
  uint32_t at;            // second product: where its rows begin in shared memory
};

// A task's rows come in stages of 16 gate and 16 up rows, long rows in stages of
// 8, in two slabs by turns: the stage after the next is requested as soon as one is used.
template <int FMT>
__global__ void __launch_bounds__(kThreads, 3) moe_up_tasks_kernel(const MoeLayerArgs a, const int32_t* ids, int most, int stage_rows, uint8_t* h8,
                                                                unsigned* status) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ TaskInfo s_task[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = a.k / kQK, parts = a.f / kHRows;
  const uint32_t rowbytes = static_cast<uint32_t>(nb) * kBB, bytes = stage_rows * rowbytes, slab = region(bytes);
  const int stages = kHRows / stage_rows;
  const UpTaskLayout l = up_task_layout(nb, kBB, most, stage_rows);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + l.recs);
  float* part = reinterpret_cast<float*>(smem + l.part);
  const int pitch = pitch_of(nb), words = kHRows * pitch;  // partials of a product of a pair
  if (tid == 0) {
    mbar_init(&bars[0], 2);
    mbar_init(&bars[1], 2);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  Table table;
  const int tasks = build_table(smem + l.total, ids, a.n_experts, a.t * a.top_k, most, table) * parts;
  auto prepare = [&](int task, int slot) {  // one thread
    const int chunk = task / parts;
    const Task x = find_task(table, a.n_experts, chunk);
    TaskInfo& to = s_task[slot];
    to.first = x.first;
    to.pairs = x.pairs;
    to.range = task - chunk * parts;
    const int64_t at = (static_cast<int64_t>(x.expert) * a.f + to.range * kHRows) * rowbytes;
    for (int m = 0; m < 2; ++m) to.src[m] = (m ? a.up : a.gate) + at;
  };
  auto fetch = [&](int slot, int stage) {  // the same thread; `stages` is even, so a stage's slab is that of its parity
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // behind the plain stores and reads of the stage before
    for (int m = 0; m < 2; ++m)
      request(smem + (2 * (stage & 1) + m) * slab, s_task[slot].src[m] + stage * bytes, bytes, &bars[stage & 1], l2_evict_first_policy());
  };
  if (tid == 0 && static_cast<int>(blockIdx.x) < tasks) {
    prepare(blockIdx.x, 0);
    fetch(0, 0);
    fetch(0, 1);
  }
  __syncthreads();
#pragma unroll 1
  for (int task = blockIdx.x, turn = 0; task < tasks; task += gridDim.x, ++turn) {
    const int slot = turn & 1;
    const TaskInfo& x = s_task[slot];
    for (int i = tid; i < x.pairs * nb * 8; i += kThreads) {
      const int c = i / (nb * 8), j = i - c * nb * 8;
      const int64_t token = table.plist[x.first + c] / a.top_k;
      fill_precord_chunk(a.q8 + (token * nb * 8 + j) * kQ8Bytes, recs + (c * nb + (j >> 3)) * kPRec, j & 7);
    }
    __syncthreads();  // the records; and everybody is done with the partials of the task before
    const bool more = task + static_cast<int>(gridDim.x) < tasks;
#pragma unroll 1
    for (int stage = 0; stage < stages; ++stage) {
      const int which = stage & 1, use = turn * (stages / 2) + (stage >> 1);  // of the slab: how often it was filled before
      const bool ok = mbar_wait(&bars[which], slot_phase(use));
      if (ok) {
        rows_dots<FMT>(2 * which * slab + low4(x.src[0] + stage * bytes), (2 * which + 1) * slab + low4(x.src[1] + stage * bytes), words, nb,
                       stage_rows, l.recs, x.pairs, l.part + 4 * stage * stage_rows * pitch, 2 * words);
      }
      if (__syncthreads_or(!ok)) {
        if (tid == 0) {
          raise_status(status, kStatusTimeout);
          // Let copies land (bounded): this stage's, and the next's, of this task or another.
          (void)mbar_wait(&bars[which], slot_phase(use));
          if (stage + 1 < stages || more) (void)mbar_wait(&bars[which ^ 1], slot_phase(turn * (stages / 2) + ((stage + 1) >> 1)));
        }
        return;
      }
      if (tid == 0) {
        if (stage + 2 < stages) {
          fetch(slot, stage + 2);
        } else if (more) {
          if (stage + 2 == stages) prepare(task + gridDim.x, slot ^ 1);
          fetch(slot ^ 1, stage + 2 - stages);
        }
      }
    }
    for (int c = warp; c < x.pairs; c += kWarps) {
      const float* of = part + c * 2 * words + lane * pitch;
      float g = 0.0f, u = 0.0f;
#pragma unroll 4
      for (int b = 0; b < nb; ++b) {
        g += of[b];
        u += of[words + b];
      }
      store_h(g, u, h8 + (static_cast<int64_t>(table.plist[x.first + c]) * parts + x.range) * kQ8Bytes);
    }
  }
}

struct DownTaskLayout {
  uint32_t slab, recs, part, total;
};
__host__ __device__ __forceinline__ DownTaskLayout down_task_layout(int nbf, int block_bytes, int rows, int pairs) {
  DownTaskLayout l;
  l.slab = 2 * region(rows * nbf * block_bytes);  // one is filled while the other is multiplied
  l.recs = l.slab;
  l.part = l.recs + pairs * nbf * kPRec * 4;
  l.total = l.part + pairs * rows * pitch_of(nbf) * 4;
  return l;
}

// y[pair][k]: the pair's product, times its weight.
template <int FMT>
__global__ void __launch_bounds__(kThreads, 3) moe_down_tasks_kernel(const MoeLayerArgs a, const int32_t* ids, const float* weights, int most,
                                                                  int rows, const uint8_t* h8, float* y, unsigned* status) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ TaskInfo s_task[2];
  const int tid = threadIdx.x;
  const int nbf = a.f / kQK, ranges = (a.k + rows - 1) / rows;
  const uint32_t rowbytes = static_cast<uint32_t>(nbf) * kBB, slab = region(rows * rowbytes);
  const DownTaskLayout l = down_task_layout(nbf, kBB, rows, most);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + l.recs);
  float* part = reinterpret_cast<float*>(smem + l.part);
  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  // The ids were complete before the first kernel let this one begin.
  Table table;
  const int tasks = build_table(smem + l.total, ids, a.n_experts, a.t * a.top_k, most, table) * ranges;
  auto prepare = [&](int task, int slot) {  // one thread
    const int chunk = task / ranges;
    const Task x = find_task(table, a.n_experts, chunk);
    TaskInfo& to = s_task[slot];
    to.first = x.first;
    to.pairs = x.pairs;
    to.range = task - chunk * ranges;
    const uint8_t* src = a.down + (static_cast<int64_t>(x.expert) * a.k + to.range * rows) * rowbytes;
    to.at = slot * slab + low4(src);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // behind the plain stores and reads of two tasks before
    request(smem + slot * slab, src, min(rows, a.k - to.range * rows) * rowbytes, &bars[slot], l2_evict_first_policy());
  };
  if (tid == 0 && static_cast<int>(blockIdx.x) < tasks) prepare(blockIdx.x, 0);
  pdl_wait();  // h is complete
  pdl_launch_dependents();
  __syncthreads();
#pragma unroll 1
  for (int task = blockIdx.x, turn = 0; task < tasks; task += gridDim.x, ++turn) {
    const int slot = turn & 1;
    const TaskInfo& x = s_task[slot];
    for (int i = tid; i < x.pairs * nbf * 8; i += kThreads) {
      const int c = i / (nbf * 8), j = i - c * nbf * 8;
      fill_precord_chunk(h8 + (static_cast<int64_t>(table.plist[x.first + c]) * nbf * 8 + j) * kQ8Bytes,
                         recs + (c * nbf + (j >> 3)) * kPRec, j & 7);
    }
    __syncthreads();  // the records; and everybody is done with the task before
    // The next task's weights and info; the barrier behind the products orders them.
    const bool more = tid == 0 && task + static_cast<int>(gridDim.x) < tasks;
    if (more) prepare(task + gridDim.x, slot ^ 1);
    const int n = min(rows, a.k - x.range * rows);
    const bool ok = mbar_wait(&bars[slot], slot_phase(turn >> 1));
    if (ok) rows_dots<FMT>(x.at, 0, 0, nbf, n, l.recs, x.pairs, l.part, n * pitch_of(nbf));
    if (__syncthreads_or(!ok)) {
      if (tid == 0) {
        raise_status(status, kStatusTimeout);
        (void)mbar_wait(&bars[slot], slot_phase(turn >> 1));  // let copies land (bounded)
        if (more) (void)mbar_wait(&bars[slot ^ 1], slot_phase((turn + 1) >> 1));
      }
      return;
    }
    for (int i = tid; i < x.pairs * n; i += kThreads) {
      const int c = i / n, p = table.plist[x.first + c];
      float v = 0.0f;
      for (int b = 0; b < nbf; ++b) v += part[i * pitch_of(nbf) + b];
      y[static_cast<int64_t>(p) * a.k + x.range * rows + i - c * n] = __ldcg(weights + p) * v;
    }
  }
}

// out = res + the slots' products in order.
__global__ void __launch_bounds__(kThreads) moe_sum_kernel(const MoeLayerArgs a, const int32_t* ids, const float* y) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= static_cast<int64_t>(a.t) * a.k) return;
  const int64_t token = at / a.k, col = at - token * a.k;
  float v = 0.0f;
#pragma unroll 4
  for (int s = 0; s < a.top_k; ++s) {
    const int64_t p = token * a.top_k + s;
    const float x = y[p * a.k + col];
    if (ids[p] >= 0) v += x;
  }
  store_out(a, at, v);
}

// ------------------------------------------------------------------- host --
int configure(const void* kern, int which) {
  static std::atomic<bool> done[10][64];  // per kernel and device (racing threads configure twice: idempotent)
  const int dev = device_info().device;
  if (dev < 0 || dev >= 64) return TQ1_ERR_CUDA;
  if (!done[which][dev].load(std::memory_order_acquire)) {
    if (!cuda_ok(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem)))) return TQ1_ERR_CUDA;
    done[which][dev].store(true, std::memory_order_release);
  }
  return TQ1_OK;
}

template <typename... Formal, typename... Actual>
int run(void (*kern)(Formal...), int64_t grid, int threads, size_t smem, cudaStream_t s, Actual... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kern, args...)) ? TQ1_OK : TQ1_ERR_CUDA;
}

template <int FMT>
int launch_pairs(const MoeLayerArgs& a, uint8_t* h8, unsigned* status, cudaStream_t s) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  const int nb = a.k / kQK, nbf = a.f / kQK;
  const UpLayout up = up_layout(nb, kBB, 1);
  // Output rows of a CTA of the second kernel: about three CTAs an SM (five
  // tokens of 8 of 128 experts of 768 x 2048, TQ2_0, 18.6 us, with two an SM 20.3, with four 22.5).
  const int64_t sms = std::max(1, device_info().num_sms);
  int64_t rows = (static_cast<int64_t>(a.k) * a.t + 3 * sms - 1) / (3 * sms);
  rows = std::min<int64_t>(64, std::max<int64_t>(4, (rows + 3) / 4 * 4));
  int slots = a.top_k;
  while (slots > 1 && down_layout(nbf, kBB, static_cast<int>(rows), slots).total > kMaxSmem / 2) --slots;
  while (rows > 4 && down_layout(nbf, kBB, static_cast<int>(rows), slots).total > kMaxSmem) rows -= 4;
  const DownLayout down = down_layout(nbf, kBB, static_cast<int>(rows), slots);
  // While every SM has two CTAs at most, twice the threads: one token of eight
  // experts of 768 x 2048 11.2 -> 10.8 us (five tokens 20.2 -> 24.1, so not there).
  const int64_t ctas = static_cast<int64_t>(a.t) * a.top_k * (a.f / kHRows);
  auto* kern = ctas <= 2 * sms ? moe_up_kernel<FMT, 2 * kThreads> : moe_up_kernel<FMT, kThreads>;
  if (configure(reinterpret_cast<const void*>(kern), ctas <= 2 * sms ? 8 + FMT : 4 * FMT) != TQ1_OK ||
      configure(reinterpret_cast<const void*>(moe_down_kernel<FMT>), 4 * FMT + 1) != TQ1_OK)
    return TQ1_ERR_CUDA;
  const int rc = run(kern, ctas, ctas <= 2 * sms ? 2 * kThreads : kThreads, up.total, s, a, h8, status);
  if (rc != TQ1_OK) return rc;
  return run(moe_down_kernel<FMT>, a.t * ((a.k + rows - 1) / rows), kThreads, down.total, s, a, static_cast<const uint8_t*>(h8),
             static_cast<int>(rows), slots, status);
}

// Whether the one form and the other have room for such rows: one pair's, and
// in the shared form four or eight rows at a time beside its table.
template <int FMT>
bool pairs_fit(int nb, int nbf) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  return up_layout(nb, kBB, 1).total <= kMaxSmem && down_layout(nbf, kBB, 4, 1).total <= kMaxSmem;
}
template <int FMT>
bool tasks_fit(int nb, int nbf, int n_experts, int pairs) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  const uint32_t table = table_bytes(n_experts, pairs);
  return up_task_layout(nb, kBB, 1, kHRows / 4).total + table <= kMaxSmem && down_task_layout(nbf, kBB, 4, 1).total + table <= kMaxSmem;
}
template <int FMT>
bool serves(int n_experts, int64_t k, int64_t f, int64_t pairs) {
  const int nb = static_cast<int>(k / kQK), nbf = static_cast<int>(f / kQK);
  return pairs_fit<FMT>(nb, nbf) || tasks_fit<FMT>(nb, nbf, n_experts, static_cast<int>(pairs));
}

// The workspace: h, and for the task kernels ids, weights and the pairs' products.
struct Workspace {
  size_t h8, ids, weights, y, total;
};
Workspace workspace(int64_t k, int64_t f, int64_t pairs) {
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  Workspace w;
  w.h8 = 0;
  w.ids = w.h8 + up(static_cast<size_t>(pairs) * (f / kQK8) * kQ8Bytes);
  w.weights = w.ids + up(static_cast<size_t>(pairs) * 4);
  w.y = w.weights + up(static_cast<size_t>(pairs) * 4);
  w.total = w.y + up(static_cast<size_t>(pairs) * k * 4);
  return w;
}

// How many experts are selected, were they selected evenly.
double used_experts(const MoeLayerArgs& a) {
  const double pairs = static_cast<double>(a.t) * a.top_k, n = a.n_experts;
  return n * (1.0 - std::pow(1.0 - 1.0 / n, pairs));
}

template <int FMT>
int launch_tasks(const MoeLayerArgs& a, uint8_t* ws, unsigned* status, cudaStream_t s) {
  constexpr int kBB = fmt_block_bytes<FMT>();
  const int nb = a.k / kQK, nbf = a.f / kQK, pairs = a.t * a.top_k;
  const Workspace w = workspace(a.k, a.f, pairs);
  const uint32_t table = table_bytes(a.n_experts, pairs);
  auto up_size = [&](int most, int stage_rows) { return up_task_layout(nb, kBB, most, stage_rows).total + table; };
  auto down_size = [&](int64_t rows, int most) { return down_task_layout(nbf, kBB, static_cast<int>(rows), most).total + table; };
  // The first product: three CTAs an SM, if four pairs have room beside stages
  // of 16 rows.  Else stages of 8 rows and three CTAs, unless two CTAs and stages
  // of 16 leave room for more pairs and experts have many (of 8 experts of 2816 x
  // 4096, 14 pairs 41 us with three CTAs and up to four pairs, 44 with two and six; 24 pairs 58 and 54).
  auto room = [&](int stage_rows, size_t smem) {  // for so many pairs
    int most = kChunk<FMT>;
    while (most > 0 && up_size(most, stage_rows) > smem) --most;
    return most;
  };
  int stage_rows = kHRows / 2, most = room(stage_rows, kThirdSmem), most_down = kChunk<FMT>;
  if (most < 4) {
    const int three = room(kHRows / 4, kThirdSmem), two = room(kHRows / 2, kHalfSmem);
    most = two;
    if (three >= 3 && (three >= two || pairs <= 2.5 * used_experts(a))) {
      stage_rows = kHRows / 4;
      most = three;
    } else if (two < 3) {
      stage_rows = kHRows / 4;
      most = std::max(1, room(stage_rows, kHalfSmem));
    }
  }
  // Rows of a task of the second product: two units a thread, or what fits.
  int64_t rows = std::min<int64_t>(a.k, std::max<int64_t>(4, 2 * kThreads / nbf / 4 * 4));
  while (rows > 4 && down_size(rows, most_down) > kThirdSmem) rows -= 4;
  while (most_down > 1 && down_size(rows, most_down) > kHalfSmem) --most_down;
  const size_t up_bytes = up_size(most, stage_rows), down_bytes = down_size(rows, most_down);
  if (configure(reinterpret_cast<const void*>(moe_up_tasks_kernel<FMT>), 4 * FMT + 2) != TQ1_OK ||
      configure(reinterpret_cast<const void*>(moe_down_tasks_kernel<FMT>), 4 * FMT + 3) != TQ1_OK)
    return TQ1_ERR_CUDA;
  int32_t* ids = reinterpret_cast<int32_t*>(ws + w.ids);
  float* weights = reinterpret_cast<float*>(ws + w.weights);
  float* y = reinterpret_cast<float*>(ws + w.y);
  int rc = run(moe_route_kernel, (a.t + kWarps - 1) / kWarps, kThreads, 0, s, a, ids, weights);
  if (rc != TQ1_OK) return rc;
  const int64_t sms = std::max(1, device_info().num_sms);
  auto grid = [&](size_t smem, int64_t tasks) {  // as many CTAs as are resident, or the most tasks there can be
    const int64_t fit = std::max<int64_t>(1, std::min<int64_t>(3, static_cast<int64_t>(228 * 1024 / (smem + 1024))));
    return std::min(fit * sms, tasks);
  };
  const int64_t active = std::min<int64_t>(pairs, a.n_experts);
  const int64_t parts = a.f / kHRows, ranges = (a.k + rows - 1) / rows;
  rc = run(moe_up_tasks_kernel<FMT>, grid(up_bytes, (active + pairs / most) * parts), kThreads, up_bytes, s, a, static_cast<const int32_t*>(ids), most, stage_rows, ws + w.h8,
           status);
  if (rc != TQ1_OK) return rc;
  rc = run(moe_down_tasks_kernel<FMT>, grid(down_bytes, (active + pairs / most_down) * ranges), kThreads, down_bytes, s, a,
           static_cast<const int32_t*>(ids), static_cast<const float*>(weights), most_down, static_cast<int>(rows),
           static_cast<const uint8_t*>(ws + w.h8), y, status);
  if (rc != TQ1_OK) return rc;
  return run(moe_sum_kernel, (static_cast<int64_t>(a.t) * a.k + kThreads - 1) / kThreads, kThreads, 0, s, a, static_cast<const int32_t*>(ids),
             static_cast<const float*>(y));
}

}  // namespace

bool moe_layer_serves(int fmt, int64_t n_experts, int64_t k, int64_t f, int64_t pairs) {
  return fmt == kFmtTq2 ? serves<kFmtTq2>(static_cast<int>(n_experts), k, f, pairs)
                        : serves<kFmtTq1>(static_cast<int>(n_experts), k, f, pairs);
}

size_t moe_layer_workspace_bytes(int64_t k, int64_t f, int64_t t, int64_t top_k) { return workspace(k, f, t * top_k).total; }

// Whether tokens that share experts share their expansion: where that saves
// 200 million weights of expanding (TQ2_0: 300 million of reading), which the two
// kernels more that it takes cost about.  Not shared and shared: 8 tokens of 8 of
// 128 experts of 768 x 2048 34 and 41 us, 16 tokens 63 and 59; 4 tokens of two of
// 8 experts of 2816 x 4096 27 and 37, 7 tokens 45.6 and 41, 12 tokens 75 and 54;
// TQ2_0 7 tokens 36 and 39, 12 tokens 59 and 49.
bool shares(const MoeLayerArgs& a, int fmt) {
  const double pairs = static_cast<double>(a.t) * a.top_k;
  const double chunks = std::max(used_experts(a), pairs / (fmt == kFmtTq2 ? kChunk<kFmtTq2> : kChunk<kFmtTq1>));
  return (pairs - chunks) * 3.0 * a.k * a.f > (fmt == kFmtTq2 ? 3e8 : 2e8);
}

// Where the rows are too long for the one form, the other has room (which the
// caller has seen to): the shared one stages 8 of them at a time, but keeps a table.
template <int FMT>
int launch_format(const MoeLayerArgs& a, uint8_t* ws, unsigned* status, cudaStream_t s) {
  const int nb = a.k / kQK, nbf = a.f / kQK;
  const bool tasks = shares(a, FMT) ? tasks_fit<FMT>(nb, nbf, a.n_experts, a.t * a.top_k) : !pairs_fit<FMT>(nb, nbf);
  return tasks ? launch_tasks<FMT>(a, ws, status, s) : launch_pairs<FMT>(a, ws, status, s);
}

int launch_moe_layer(const MoeLayerArgs& a, int fmt, void* ws, unsigned* status, cudaStream_t s) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  return fmt == kFmtTq2 ? launch_format<kFmtTq2>(a, w, status, s) : launch_format<kFmtTq1>(a, w, status, s);
}

}  // namespace tq1
