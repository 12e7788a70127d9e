// attn_tile.cu -- attention over the paged cache on the 5th-generation tensor
// cores, for calls with many rows per kv head (prompt chunks).
//
// The mathematics and the division of work are attn.cu's and kv.cuh's; here a
// tile is 128 rows (or two of them) and a block 128 keys:
//   S = Q K^T   tcgen05.mma 128 x 128 x 16, both operands in shared memory
//   P = exp2(scale log2e S - m), 16 bits, written over S in tensor memory
//   O += P V    tcgen05.mma 128 x d x 16, P from tensor memory, V from shared
//               memory as it lies in the cache (keys by elements: the operand's
//               other major order), O in tensor memory
//
// Bound: the tensor pipe.  Per 128 x 128 keys it takes 8 d cycles for both
// products (4096 multiply-adds a cycle), the exponentials 512; so two streams
// of (S, P, O), one warp group each, take turns: while one's weights are
// formed the tensor pipe does the other's products.  What it comes to is the
// latency of a stream's chain, which one block after the other goes through:
// at d = 128 some 1400 cycles for a block's weights (450 to read the scores
// and find the maximum, 800 for the exponentials, 110 to store them), 1024 in
// the tensor pipe and 400 between the roles, against 2048 of tensor work for
// both streams.  S and P of a second block per stream would break the chain;
// the two O leave no tensor memory for them.
// 4096 tokens on 12288 keys, 40/8 heads of 128: 580 us call after call, at the
// power limit's lower clock, 1.48 PFLOP/s; 550 us in a short run.  A ragged
// batch (1 to 1463 tokens, 24/8 heads of 64, window 1024): 45.9 us in a graph,
// 47.7 a call, of which 5 pass before the first scores.
//   PAIR:  a tile has two times 128 rows, a stream each, and both read the
//          same keys (a chunk with more than 128 rows per kv head)
//   else:  a tile has 128 rows; the streams take every other block and are
//          joined at the tile's end (fewer rows: the cache's length is what is
//          left to share out)
// Rows are (token, query head of the group), token by token: a tile holds
// floor(128 / group) whole tokens, so the queries of a tile are one box of q,
// and every key is read once for the whole group.
//
// Rescaling: O stays relative to a reference maximum that is moved (and O
// with it, through registers) only when a row's maximum has grown by more than
// 2^8 over it; weights up to 2^8 lose nothing, 16-bit floats being relative.
//
// Roles: warp 0 the matrix instructions, warp 1 the copies (TMA, a box per
// page and 64 elements, 128-byte swizzle), warp 2 walks the CTA's tiles for all
// of them, warps 4-7 and 8-11 the two streams' weights (a thread a row).
// Keys at or past a sequence's length are not read at all where a whole page
// of them is; values that no token of the call sees are overwritten with
// zeros in shared memory before the second product: a weight of zero would not
// silence a NaN there.
//
// Every wait is bounded; the first that runs out sets an abort flag that
// releases the others, and TQ1_ERR_TIMEOUT is raised.
#include <atomic>
#include <type_traits>

#include "../../include/tq1.h"
#include "kv.cuh"
#include "tcgen05.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

constexpr int kTThreads = 384, kMmaWarp = 0, kLoadWarp = 1, kPlanWarp = 2;  // warp 3 makes the first warp group whole
// Registers per thread: 384 x 168 at launch = 2 x 128 x 208 + 128 x 88.
constexpr int kWeightRegs = 208, kOtherRegs = 88;
constexpr int kTRows = 128;   // rows of a stream (tensor-memory lanes)
constexpr int kTShift = 7, kTBlock = 1 << kTShift;  // keys of a block
constexpr float kMoveAt = 8.0f;  // log2 of how far a row's maximum may outgrow its reference
// log2 of what the weights are formed times (it cancels in O / l): with it the
// largest weight there can be, 2^kMoveAt of the reference's, is 2^15, which
// fp16 just holds; so weights down to 2^-21 of the reference's are whole and
// nothing is zero above 2^-32, where without it those are 2^-14 and 2^-25.
// bf16 has fp32's range.
template <typename T>
constexpr float kTLift = std::is_same<T, __half>::value ? 15.0f - kMoveAt : 0.0f;

template <int D, bool PAIR>
struct TileCfg {
  static constexpr uint32_t kHalf = kTBlock * 128;             // 64 elements of 128 rows
  static constexpr uint32_t kTile = (D / 64) * kHalf;          // 128 rows of q, keys or values
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr uint32_t kStatic = PAIR ? 1536 : 3584;      // at most: barriers, segments, the streams' join
  static constexpr int kRing = static_cast<int>((232448 - kStatic - 1024) / kTile) - kQTiles;
  static constexpr uint32_t kSmem = (kQTiles + kRing) * kTile + 1024;
  // A stream's next block.  Blocks of keys are copied so many blocks ahead of
  // their values, so a segment of n blocks fills its ring slots in the order
  //   PAIR: K0 V0 K1 V1 K2 ...      else: K0 K1 V0 K2 V1 K3 V2 ...
  static constexpr int kStep = PAIR ? 1 : 2;
  static __device__ __forceinline__ uint32_t value_slot(int i, int n) { return PAIR ? 2 * i + 1 : i + min(i + 2, n); }
  static constexpr uint32_t kO = 256;  // tensor-memory columns: S of stream s at 128 s, O at kO + s D
};

struct TileKernelArgs {
  KvCache c;
  KvBatch b;
  AttnArgs a;
  TilePlan plan;
  Part* parts;
  float* slots;
  unsigned* status;
  int stream_rows, stream_tokens;  // rows and tokens of a stream: floor(128 / group) tokens
  int box_keys;                    // keys of a copied box
  int out32;                       // output rows begin on 32-byte boundaries
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  bool there = false;
#pragma unroll 1
  for (int i = 0; i < 64 && !there; ++i) there = mbar_try_wait(bar, parity);
  if (!there) there = wait_or_abort(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, there);  // the warp's lanes leave together, with one answer
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A wait that ends in any case and says nothing: the phase completed, or
// another role has aborted, or ~2 s went by, in which case it sets the flag
// itself.  Whoever goes on after an abort works on what is there; the call
// reports TQ1_ERR_TIMEOUT.  One block of instructions to the compiler, which
// sees no branch in it.
__device__ __forceinline__ void wait_soft(uint64_t* bar, uint32_t parity, int* abort_flag) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u64 t, t0;\n\t.reg .u32 f;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t0, %%globaltimer;\n\t"
      "add.u64 t0, t0, %3;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.u32 f, [%2];\n\t"
      "setp.ne.u32 q, f, 0;\n\t"
      "@q bra DONE;\n\t"
      "mov.u64 t, %%globaltimer;\n\t"
      "setp.lt.u64 q, t, t0;\n\t"
      "@q bra AGAIN;\n\t"
      "st.volatile.shared.u32 [%2], 1;\n\t"
      "DONE:\n\t}" ::"r"(smem_addr(bar)),
      "r"(parity), "r"(smem_addr(abort_flag)), "l"(kWaitLimitNs)
      : "memory");
}
// The value of lane 0, which the compiler then knows to be every lane's.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Keys by elements (K order down the rows, 64 elements of N along a row):
// the operand's N-major order, 128-byte swizzle.  Blocks of 64 elements lie
// `lead` bytes apart, groups of eight keys 1024.
__device__ __forceinline__ uint64_t umma_desc_nmajor(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// D (TMEM) += A (shared memory) * B (shared memory).
__device__ __forceinline__ void umma_ss(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Uses of v stay behind the wait that precedes this.
__device__ __forceinline__ void hold(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (a.x * b + c, a.y * b + c)
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  uint64_t r, x, y, z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(z) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}

// A thread's 32 bytes of an output row, in one store where the rows allow it:
// the warp's 32 rows are 32 lines, and whole sectors take half as long as
// halves (ragged mix 47.5 -> 46.6 us, 64 chunks of 20 to 200 tokens 52.6 -> 51.5).
__device__ __forceinline__ void store_32bytes(void* dst, const uint32_t (&w)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// One tile's share of this CTA, as the planning warp hands it to the others.
struct Segment {
  int head, seq, q0, len;  // kv head; sequence, its first token and its length
  int pos0;                // position of its first token
  int tok0, rows;          // first token and rows of the tile
  int first_key, todo;     // blocks of the tile done here (0: no more segments)
  int lo;                  // first key that some token of the sequence's sees
  int hi;                  // keys [.., hi) are seen by some row
  int starts, ends;        // whether they include the tile's first, last block
  int empty;               // no row sees a key: nothing is read
  int last_cta;            // the CTA that does its last block
};
constexpr int kSegs = 4;            // segments in flight
constexpr int kSegReaders = 8 + 2;  // warps that read them

}  // namespace

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(kTThreads, 1)
    attn_tile_kernel(const TileKernelArgs k, const __grid_constant__ CUtensorMap tmq,
                     const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using C = TileCfg<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[C::kRing], empty[C::kRing];
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], swap, drained;
  __shared__ __align__(8) uint64_t seg_full[kSegs], seg_empty[kSegs];
  __shared__ Segment s_seg[kSegs];
  __shared__ float s_ml[2][2][kTRows];  // [stream][m, l][row]: the streams' join
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const uint32_t raw = smem_addr(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (sbase - raw);
  const uint32_t q_at = sbase, ring_at = sbase + C::kQTiles * C::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_full[s], 1);
    }
    mbar_init(&swap, 8);
    mbar_init(&drained, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], kSegReaders);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns were asked for: they begin at column 0
  pdl_wait();
  pdl_launch_dependents();
  const Start st = find_start<kTThreads>(k.plan, k.b, k.c.n_kv, cta, ctas, reinterpret_cast<int64_t*>(sm));
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copies below write where the search wrote
  __syncthreads();
  if (tid < 2) k.parts[2 * cta + tid].rows = 0;
  if (st.bad && cta == 0 && tid == 0) raise_status(k.status, kStatusBadId);
  __syncthreads();
  // The next segment, for one of the reading warps; false after an abort.
  uint32_t seg_at = 0;
  Segment g;
  auto next_segment = [&]() {
    const uint32_t i = seg_at % kSegs;
    if (!wait_all(&seg_full[i], (seg_at / kSegs) & 1u, abort_flag)) return false;
    g = s_seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[i]);
    ++seg_at;
    return true;
  };

  // The weights' branch is the last in the text: where the roles' loops come
  // to lie is worth 2% (chunk, call after call: 600 us with it first, 586 so).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
      // ----------------------------------------------------------- MMA --
      // In a step (a block's second product and the first product kStep
      // blocks on) the streams take turns; issued from a warp each, their
      // instructions would interleave and both streams' products finish late
      // (4096 tokens on 12288 keys, 40/8 heads of 128: 670 us for 560).
      //
      // The whole warp walks the loop without a branch on what a lane has
      // seen (wait_soft), and one lane issues: addresses and descriptors are
      // then the same in all lanes to the compiler too, which keeps them in
      // the uniform registers that the instructions take.
      constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t kIdS = (1u << 4) | (kType << 7) | (kType << 10) | ((kTBlock >> 3) << 17) | ((kTRows >> 4) << 24);
      constexpr uint32_t kIdO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((D >> 3) << 17) | ((kTRows >> 4) << 24);
      const bool lead = elect_one();
      const uint64_t qd0 = umma_desc_sw128(q_at), kd0 = umma_desc_sw128(ring_at);
      const uint64_t vd0 = umma_desc_nmajor(ring_at, C::kHalf);
      uint32_t pph = 0, qph = 0;   // phases of p_full (a bit per stream) and q_full
      uint32_t ri = 0, rph = 0;    // ring slot to be consumed next, its phase
      auto step = [&]() {
        if (++ri == C::kRing) {
          ri = 0;
          rph ^= 1u;
        }
      };
      auto product_s = [&](int s, uint32_t slot) {
        const uint64_t qd = qd0 + (((PAIR ? s : 0) * C::kTile) >> 4), kd = kd0 + ((slot * C::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * C::kHalf + (ks & 3) * 32u) >> 4;
          umma_ss(tmem + 128 * s, qd + off, kd + off, kIdS, ks > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[s]);
      };
      // Keys in steps of 16, [from, steps) of them.
      auto product_o = [&](int s, uint32_t slot, int from, int steps, uint32_t keep) {
        const uint32_t s_col = tmem + 128 * s, o_col = tmem + C::kO + s * D;
        const uint64_t vd = vd0 + ((slot * C::kTile) >> 4);
        if (from == 0 && steps == kTBlock / 16) {
#pragma unroll
          for (int ks = 0; ks < kTBlock / 16; ++ks)
            umma_ts(o_col, s_col + 8 * ks, vd + ((ks * 2048u) >> 4), kIdO, ks > 0 ? 1u : keep);
        } else {
          for (int ks = from; ks < steps; ++ks)
            umma_ts(o_col, s_col + 8 * ks, vd + ((ks * 2048u) >> 4), kIdO, ks > from ? 1u : keep);
        }
      };
      for (uint32_t at = 0;; ++at) {
        wait_soft(&seg_full[at % kSegs], (at / kSegs) & 1u, &s_abort);
        const int n = uniform(*abort_flag ? 0 : s_seg[at % kSegs].todo), none = uniform(s_seg[at % kSegs].empty);
        const int first_key = uniform(s_seg[at % kSegs].first_key), hi = uniform(s_seg[at % kSegs].hi);
        const int lo = uniform(s_seg[at % kSegs].lo);
        if (lead) mbar_arrive(&seg_empty[at % kSegs]);
        if (n == 0) break;
        if (none) continue;
        wait_soft(&q_full, qph, &s_abort);
        qph ^= 1u;
#pragma unroll
        for (int i = 0; i < C::kStep; ++i) {
          if (i >= n) break;
          wait_soft(&full[ri], rph, &s_abort);
          tc_fence_after();
          if (lead) {
            product_s(PAIR ? 0 : i, ri);
            if (PAIR) product_s(1, ri);
            umma_commit(&empty[ri]);
          }
          step();
        }
        for (int i = 0; i < n; ++i) {
          const bool more = i + C::kStep < n;
          // The last first product is on its way.
          if (lead && (i + C::kStep == n || (i == 0 && n < C::kStep))) umma_commit(&q_empty);
          const int key0 = first_key + i * kTBlock;
          const int steps = (min(kTBlock, hi - key0) + 15) >> 4, from = max(0, lo - key0) >> 4;
          const uint32_t slot = ri, sph = rph;
          step();
          const uint32_t nslot = ri, nph = rph;
          if (more) step();
          wait_soft(&full[slot], sph, &s_abort);
          if (more) wait_soft(&full[nslot], nph, &s_abort);
#pragma unroll
          for (int u = 0; u < (PAIR ? 2 : 1); ++u) {
            const int s = PAIR ? u : (i & 1);
            wait_soft(&p_full[s], (pph >> s) & 1u, &s_abort);
            pph ^= 1u << s;
            tc_fence_after();
            if (lead) {
              product_o(s, slot, from, steps, i >= C::kStep ? 1u : 0u);
              if (u == (PAIR ? 1 : 0)) umma_commit(&empty[slot]);
              if (more) {
                product_s(s, nslot);
                if (u == (PAIR ? 1 : 0)) umma_commit(&empty[nslot]);
              } else {
                umma_commit(&o_full[s]);
              }
            }
          }
        }
      }
      // After an abort, let the products already issued finish (bounded).
      __syncwarp();
      if (*abort_flag) {
        if (lead) umma_commit(&drained);
        (void)mbar_wait(&drained, 0);
      }
    } else if (warp == kLoadWarp) {
      // --------------------------------------------------------- copies --
      uint32_t at = 0, segs = 0;  // ring slots filled, segments read
      bool ok = true;
      const int boxes = kTBlock / k.box_keys;  // of a block
      const int half = lane & (D / 64 - 1), box = lane / (D / 64);
      // The page of this lane's box of the block from key0 on: -1 (read as
      // zeros) where the table names none, -2 past the sequence's end and
      // before the window of its first token (whose page may be gone): not
      // read, as no row of the call sees it.
      auto page_of = [&](int key0) {
        const int key = key0 + box * k.box_keys;
        if (box >= boxes || key >= g.len || key + k.box_keys <= g.lo) return -2;
        const int id = k.b.table[static_cast<int64_t>(g.seq) * k.b.max_pages + (key >> k.c.page_shift)];
        if (id >= 0 && id < k.c.n_pages) return id;
        raise_status(k.status, kStatusBadId);
        return -1;
      };
      auto copy = [&](const CUtensorMap* map, int key0, int page) {
        const uint32_t slot = at % C::kRing;
        if (!(ok = wait_all(&empty[slot], ((at / C::kRing) & 1u) ^ 1u, abort_flag))) return false;
        const uint32_t live = __ballot_sync(0xffffffffu, page != -2);
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], __popc(live) * k.box_keys * 128);
        __syncwarp();
        if (page != -2)
          tma_load_4d(ring_at + slot * C::kTile + half * C::kHalf + box * k.box_keys * 128, map, 64 * half,
                      (key0 + box * k.box_keys) & (k.c.page_size - 1), g.head, page, &full[slot]);
        ++at;
        return true;
      };
      while (ok && next_segment() && g.todo > 0) {
        if (g.empty) continue;
        int page[C::kStep];
#pragma unroll
        for (int i = 0; i < C::kStep; ++i) page[i] = i < g.todo ? page_of(g.first_key + i * kTBlock) : -2;
        if (!(ok = wait_all(&q_empty, (segs & 1u) ^ 1u, abort_flag))) break;
        if (lane == 0) mbar_arrive_expect_tx(&q_full, C::kQTiles * (D / 64) * k.stream_rows * 128);
        __syncwarp();
        if (lane < C::kQTiles * (D / 64)) {
          const int qs = lane / (D / 64), qhalf = lane & (D / 64 - 1);
          tma_load_3d(q_at + qs * C::kTile + qhalf * C::kHalf, &tmq, 64 * qhalf, g.head * k.plan.group,
                      g.q0 + g.tok0 + qs * k.stream_tokens, &q_full);
        }
        ++segs;
        for (int i = 0; i < C::kStep && i < g.todo && ok; ++i) copy(&tmk, g.first_key + i * kTBlock, page[i]);
        for (int i = 0; i < g.todo && ok; ++i) {
          const int next = i + C::kStep, key = g.first_key + i * kTBlock;
          const int np = next < g.todo ? page_of(g.first_key + next * kTBlock) : -2;
          if (!copy(&tmv, key, page[0])) break;
          if (next < g.todo && !copy(&tmk, g.first_key + next * kTBlock, np)) break;
#pragma unroll
          for (int j = 0; j + 1 < C::kStep; ++j) page[j] = page[j + 1];
          page[C::kStep - 1] = np;
        }
      }
      // Copies still in flight must land before the CTA leaves.
      if (lane == 0 && *abort_flag) {
        for (uint32_t i = at > C::kRing ? at - C::kRing : 0; i < at; ++i)
          (void)mbar_wait(&full[i % C::kRing], (i / C::kRing) & 1u);
        if (segs) (void)mbar_wait(&q_full, (segs - 1) & 1u);
      }
    } else if (warp == kPlanWarp) {
      // ----------------------------------------------------------- plan --
      int head = st.head, seq = st.seq, tile = st.tile, blk = st.block;
      int64_t left = st.units, unit = st.first;
      Seq sq = st.sq;
      for (bool more = true; more; ++seg_at) {
        g = Segment{};
        more = left > 0;
        if (more) {
          int fb, nb;
          tile_blocks(k.plan, sq, tile, fb, nb);
          const int row0 = tile * k.plan.rows;
          g.head = head;
          g.seq = seq;
          g.q0 = sq.q0;
          g.len = sq.len;
          g.pos0 = sq.len - sq.n;
          g.tok0 = row0 / k.plan.group;
          g.rows = min(k.plan.rows, sq.n * k.plan.group - row0);
          g.first_key = (fb + blk) * kTBlock;
          g.todo = static_cast<int>(min(static_cast<int64_t>(nb - blk), left));
          const int end = row0 + g.rows;
          g.hi = k.plan.causal ? min(sq.len, g.pos0 + (end - 1) / k.plan.group + 1) : sq.len;
          g.lo = k.plan.window ? max(0, g.pos0 - k.plan.window + 1) : 0;
          g.empty = g.hi <= (k.plan.window ? max(0, g.pos0 + g.tok0 - k.plan.window + 1) : 0);
          g.starts = blk == 0;
          g.ends = blk + g.todo == nb;
          if (g.starts && !g.ends) g.last_cta = share_of(st.work, st.used, unit + nb - 1);
        }
        const uint32_t i = seg_at % kSegs;
        if (!wait_all(&seg_empty[i], ((seg_at / kSegs) & 1u) ^ 1u, abort_flag)) break;
        if (lane == 0) {
          s_seg[i] = g;
          mbar_arrive(&seg_full[i]);
        }
        __syncwarp();
        if (more) {
          left -= g.todo + st.cost;
          unit += g.todo + st.cost;
          if (left > 0) {
            next_tile(k.plan, k.b, head, seq, tile, sq);
            blk = 0;
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------- weights --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWeightRegs));
    const int s = (warp >> 2) - 1, row = tid & (kTRows - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t st_at = tmem + lanes + 128 * s, o_at = tmem + lanes + C::kO + s * D;
    const float sc = k.a.scale * kLog2e;
    uint32_t done = 0;   // blocks this stream has done, over all segments
    uint32_t oph = 0;    // phase of o_full
    uint32_t base_slot = 0;  // ring slots of the segments before
    uint32_t swaps = 0;  // phases of `swap` passed
    bool ok = true;
    // This thread's row: its place in every tile (whole tokens, so its token
    // and head in the tile are always the same).
    const int trow = PAIR ? s * k.stream_rows + row : row;
    const int ttok = trow / k.plan.group, thead = trow - ttok * k.plan.group;
    for (bool first_seg = true; ok; first_seg = false) {
      if (!next_segment() || g.todo == 0) break;
      // The keys [lo, hi) that it sees.  Lanes past the stream's rows (or the
      // sequence's) compute on what lies in shared memory and store nothing.
      const bool there = row < k.stream_rows && trow < g.rows;
      const int tok = g.tok0 + ttok, qh = g.head * k.plan.group + thead;
      int lo = 0, hi = 0x7fffffff;
      if (there) {
        const int pos = g.pos0 + tok;
        hi = k.plan.causal ? min(g.len, pos + 1) : g.len;
        lo = k.plan.window ? max(0, pos - k.plan.window + 1) : 0;
      }
      float m = -INFINITY, l = 0.0f;  // the row's reference maximum (of S) and its sum
      if (!g.empty) {
        for (int i = PAIR ? 0 : s; i < g.todo; i += PAIR ? 1 : 2) {
          const int key0 = g.first_key + i * kTBlock;
          if (!wait_all(&s_full[s], done & 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld<32>(st_at + 32 * c, v[c]);
          wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) hold(v[c]);
          if (__any_sync(0xffffffffu, lo > key0 || hi - kTBlock < key0)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int a = min(max(lo - key0 - 32 * c, 0), 32), b = min(max(hi - key0 - 32 * c, 0), 32);
              const uint32_t seen = (b == 32 ? ~0u : (1u << b) - 1u) & (a == 32 ? 0u : ~0u << a);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(seen & (1u << j))) v[c][j] = 0xff800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
            for (int j = 2; j < 32; j += 2)
              mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(v[c][j])), __uint_as_float(v[c][j + 1]));
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool opening = i < 2 && (!PAIR || i == 0);  // nothing in O yet
          if (opening) {
            m = mt;
          } else {
            const bool move = mt > m && (mt - m) * sc > kMoveAt;
            if (__any_sync(0xffffffffu, move)) {
              float keep = 1.0f;
              if (move) {
                keep = exp2_fast((m - mt) * sc);
                m = mt;
                l *= keep;
              }
              // O is at rest: the block before was added to it ahead of this S.
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld<32>(o_at + 32 * c, o);
                wait_ld();
                hold(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                tmem_st32(o_at + 32 * c, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.0f : kTLift<T> - m * sc;  // no key seen yet: all weights are exp2(-inf) = 0
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // The weights enter the second product as 16-bit numbers of V's
            // type (the instruction wants one type); their sum stays fp32.
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int c = 2 * h + (j >> 4), e = 2 * (j & 15);
              float2 x = fma2(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc, base);
              x.x = exp2_fast(x.x);
              x.y = exp2_fast(x.y);
              sum[j & 1] = add2(sum[j & 1], x);
              p[j] = pack2<T>(x.x, x.y);
            }
            tmem_st32(st_at + 32 * h, p);
          }
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
          // Values that no token of the call sees (before the window of the
          // sequence's first, or past its end, within the first and the last
          // 16 that are multiplied) are zeroed by the first stream that reads
          // them.  Their ring slot's use before this one was over before this
          // S began, and this one is not without p_full: the phase waited for
          // is the only one it can be.
          const int below = g.lo - key0, from = g.len - key0, upto = (min(kTBlock, g.hi - key0) + 15) & ~15;
          if ((below > 0 || from < upto) && (!PAIR || s == 0)) {
            const uint32_t at = base_slot + C::value_slot(i, g.todo), slot = at % C::kRing;
            if (!(ok = wait_all(&full[slot], (at / C::kRing) & 1u, abort_flag))) break;
            uint8_t* const values = sm + (ring_at - sbase) + slot * C::kTile;
            auto zero = [&](int r0, int r1) {
              for (int e = row; e < (r1 - r0) * (D / 8); e += kTRows) {
                const int r = r0 + e / (D / 8), c = e % (D / 8);
                *reinterpret_cast<uint4*>(values + (c >> 3) * C::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
            };
            if (below > 0) zero(below & ~15, below);
            if (from < upto) zero(from, upto);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[s]);
          ++done;
        }
        if (!ok) break;
        base_slot += 2 * g.todo;
      }
      const bool mine = !g.empty && (PAIR || s < g.todo);  // this stream's O holds something
      if (mine) {
        if (!wait_all(&o_full[s], oph, abort_flag)) break;
        oph ^= 1u;
        tc_fence_after();
      }
      // Out: the row over its sum, or, of a tile that others share, the row
      // as it is; zero where it sees nothing, whatever the values are that
      // other rows see (its weights of zero did not silence a NaN).  Two
      // streams on one tile first tell each other their m and l; then each
      // does half the columns of both.
      float mrow = m == -INFINITY ? m : m * sc, lrow = l, f0 = l == 0.0f ? 0.0f : 1.0f, f1 = 0.0f;
      if (!PAIR) {
        s_ml[s][0][row] = mrow;
        s_ml[s][1][row] = l;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&swap);
        if (!wait_all(&swap, swaps & 1u, abort_flag)) break;
        ++swaps;
        tc_fence_after();
        const float m0 = s_ml[0][0][row], m1 = s_ml[1][0][row];
        mrow = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.0f : exp2f(m0 - mrow);
        f1 = m1 == -INFINITY ? 0.0f : exp2f(m1 - mrow);
        lrow = f0 * s_ml[0][1][row] + f1 * s_ml[1][1][row];
      }
      const bool whole = g.starts && g.ends;
      const int slot = first_seg ? 2 * cta : 2 * cta + 1;
      float* out = k.slots + slot * join_slot_floats(k.plan.rows, D);
      const float inv = lrow > 0.0f ? 1.0f / lrow : (lrow == 0.0f ? 0.0f : lrow);
      const int64_t at = static_cast<int64_t>(g.q0 + tok) * k.a.ldo + static_cast<int64_t>(qh) * D;
      constexpr int kCols = PAIR ? D : D / 2;
#pragma unroll 1
      for (int c = 0; c < kCols / 32; ++c) {
        const int col = (PAIR ? 0 : s * kCols) + 32 * c;
        float x[32];
        if (g.empty) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.0f;
        } else {
          uint32_t o[32];
          tmem_ld<32>(tmem + lanes + C::kO + (PAIR ? s * D : 0) + col, o);
          wait_ld();
          hold(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = f0 == 0.0f ? 0.0f : f0 * __uint_as_float(o[j]);
          if (!PAIR && g.todo > 1) {
            tmem_ld<32>(tmem + lanes + C::kO + D + col, o);
            wait_ld();
            hold(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] += f1 == 0.0f ? 0.0f : f1 * __uint_as_float(o[j]);
          }
        }
        if (!there) continue;
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(out + slot_o(k.plan.rows, trow, col + j)) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        } else if (k.a.out_f32) {
          float* dst = static_cast<float*>(k.a.out) + at + col;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(x[j + e] * inv);
            store_32bytes(dst + j, w, k.out32);
          }
        } else {
          uint16_t* dst = static_cast<uint16_t*>(k.a.out) + at + col;
#pragma unroll
          for (int j = 0; j < 32; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack2<T>(x[j + 2 * e] * inv, x[j + 2 * e + 1] * inv);
            store_32bytes(dst + j, w, k.out32);
          }
        }
      }
      if (!whole) {
        if (there && (PAIR || s == 0)) {
          out[trow] = mrow;
          out[((k.plan.rows + 3) & ~3) + trow] = lrow;
        }
        if (tid == 128 && g.starts) k.parts[slot] = Part{g.head, g.q0, g.tok0 * k.plan.group, g.rows, g.last_cta, {}};
      }
      if (!PAIR) {
        // The other stream has read this one's O and s_ml before either goes on.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&swap);
        if (!wait_all(&swap, swaps & 1u, abort_flag)) break;
        ++swaps;
        tc_fence_after();
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) raise_status(k.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

namespace {

bool make_tensor_map(CUtensorMap* map, int dtype, int rank, const void* base, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool PAIR>
int launch_cfg(const TileKernelArgs& k, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
               cudaStream_t s) {
  using C = TileCfg<D, PAIR>;
  const DeviceInfo& di = device_info();
  static std::atomic<bool> configured[64];  // per device (racing threads configure twice: idempotent)
  if (di.device < 0 || di.device >= 64) return TQ1_ERR_CUDA;
  if (C::kSmem + C::kStatic > di.max_smem_optin) return TQ1_ERR_UNSUPPORTED;
  if (!configured[di.device].load(std::memory_order_acquire)) {
    if (!cuda_ok(cudaFuncSetAttribute(attn_tile_kernel<T, D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(C::kSmem))))
      return TQ1_ERR_CUDA;
    configured[di.device].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, attn_tile_kernel<T, D, PAIR>, k, tmq, tmk, tmv)) ? TQ1_OK : TQ1_ERR_CUDA;
}

}  // namespace

int attn_tile_rows(int group, bool pair) { return (kTRows / group) * group * (pair ? 2 : 1); }

int launch_attn_tile(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool pair, int ctas, Part* parts,
                     float* slots, unsigned* status, cudaStream_t s) {
  const int group = a.n_q / c.n_kv, tokens = kTRows / group;
  // Heads or pages that are all the same one: not a tensor map's strides.
  if ((c.n_kv > 1 && c.head_stride == 0) || (c.n_pages > 1 && c.page_stride == 0)) return TQ1_ERR_UNSUPPORTED;
  TileKernelArgs k = {};
  k.c = c;
  k.b = b;
  k.a = a;
  k.plan = {Divisor(attn_tile_rows(group, pair)), Divisor(group), a.causal, a.window, kTShift};
  k.parts = parts;
  k.slots = slots;
  k.status = status;
  k.stream_rows = tokens * group;
  k.stream_tokens = tokens;
  k.box_keys = c.page_size < kTBlock ? c.page_size : kTBlock;
  const int64_t out_row = a.ldo * (a.out_f32 ? 4 : 2);
  k.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && out_row % 32 == 0;
  CUtensorMap tmq, tmk, tmv;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(a.n_q), static_cast<cuuint64_t>(b.t)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.d) * 2, static_cast<cuuint64_t>(a.ldq) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tokens)};
    if (!make_tensor_map(&tmq, c.dtype, 3, a.q, dims, strides, box)) return TQ1_ERR_UNSUPPORTED;
  }
  {
    // A dimension of one element is never stepped along; its stride may then
    // be anything in the caller's hands and is replaced by a valid one.
    const int64_t row = c.slot_stride * 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.n_kv), static_cast<cuuint64_t>(c.n_pages > 0 ? c.n_pages : 1)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(c.n_kv > 1 ? c.head_stride * 2 : row),
                                   static_cast<cuuint64_t>(c.n_pages > 1 ? c.page_stride * 2 : row)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(k.box_keys), 1, 1};
    if (!make_tensor_map(&tmk, c.dtype, 4, c.k, dims, strides, box)) return TQ1_ERR_UNSUPPORTED;
    if (!make_tensor_map(&tmv, c.dtype, 4, c.v, dims, strides, box)) return TQ1_ERR_UNSUPPORTED;
  }
#define TQ1_TILE(T, D) (pair ? launch_cfg<T, D, true>(k, tmq, tmk, tmv, ctas, s) : launch_cfg<T, D, false>(k, tmq, tmk, tmv, ctas, s))
  if (c.d == 128) return c.dtype == kBf16 ? TQ1_TILE(__nv_bfloat16, 128) : TQ1_TILE(__half, 128);
  return c.dtype == kBf16 ? TQ1_TILE(__nv_bfloat16, 64) : TQ1_TILE(__half, 64);
#undef TQ1_TILE
}

}  // namespace tq1
