// attn.cu -- attention of each sequence's newest tokens over its paged cache,
// few rows per kv head (decode steps).
//
//   O[i] = sum_j p_ij V[j],  p_ij = exp(x_ij - m_i) / l_i,  x_ij = scale q_i . K[j]
//
// over the keys j that row i sees.  One pass over the cache with a running
// maximum m and sum l per row: adding keys with a larger maximum m' rescales
// what is there by exp(m - m').  Work is divided over CTAs as kv.cuh says; a
// tile is 16 rows (tokens x query heads of one kv head) and a block 128 keys,
// of which each of the CTA's eight warps does 16.
//
// Bound: HBM, every visible key and value read once (4 d bytes per key and
// kv head, for up to 16 rows).  So the warps are independent: each copies its
// own keys and values (16-byte asynchronous copies into a ring of its own,
// several blocks ahead) and keeps its own m, l and O; nothing in the loop
// waits for another warp.  The products run on mma.sync (16 x 8 x 16): d / 4
// instructions per 16 keys and warp, far from a limit here, where a
// 128-row tensor-core tile would be at most 1/8 full.
// 64 sequences of 223 000 keys in all, 40/8 heads of 128: 144 us, 6.4 TB/s;
// one of 131 071, 32/4 heads: 49 us, 5.5 TB/s (the median CTA is done at
// 38 us, the last at 44: the SMs' shares of the bandwidth are not equal, and
// finer shares cost more in starts than they even out: 65 us with four per
// SM); one of 777: 8 us, the latency of two launches.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/tq1.h"
#include "kv.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

constexpr int kAWarps = 8, kAThreads = 32 * kAWarps;
constexpr int kAShift = 7;                // a block is 128 keys
constexpr int kARows = 16;                // rows of a tile (one m16 operand)
constexpr int kWarpKeys = 16;             // keys of a block per warp
constexpr int kABlock = kWarpKeys * kAWarps;
static_assert(kABlock == 1 << kAShift, "a warp does 16 keys of every block");

template <int D>
struct WarpCfg {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kTile = kWarpKeys * D * 2;           // one warp's keys (or values) of a block
  static constexpr uint32_t kRing = kAWarps * kStages * 2 * kTile;
  // Behind the ring, for the joining of the warps: m and l of all their rows,
  // O of eight rows at a time.
  static constexpr uint32_t kJoin = kAWarps * (2 * kARows + 8 * D) * 4;
  static constexpr uint32_t kSmem = kRing + kJoin;
  static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// log2 of what the weights are formed times, so that their 16-bit form spans
// as much below the largest as the type can hold: it cancels in O / l.  In
// fp16, weights from 1 down would be subnormal below 2^-14 and zero below
// 2^-25, while l counts them (4000 keys with weights of e^-17 to e^-20 behind
// 16 of weight 1: an output that is theirs came out 10 to 16% small); times
// 2^15 they are whole down to 2^-29.  bf16 has fp32's range.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 15.0f : 0.0f;

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

}  // namespace

namespace {

// A tile's share of this CTA.
struct WarpTile {
  int head, seq, tile, blk, nb, todo;  // blocks [blk, blk + todo) of the tile's nb
  int key0;                            // this warp's keys: key0, key0 + 128, ...
  int lo, hi;                          // keys that some row sees
  Seq sq;
};

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kAThreads, 1)
    attn_warp_kernel(const KvCache c, const KvBatch b, const AttnArgs a, const TilePlan plan, Part* parts, float* slots,
                     unsigned* status) {
  using C = WarpCfg<D>;
  constexpr int kAhead = C::kStages - 1;  // steps requested before the one being done
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int g = lane >> 2, qd = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  const Start st = find_start<kAThreads>(plan, b, c.n_kv, cta, ctas, reinterpret_cast<int64_t*>(smem));
  __syncthreads();
  if (tid < 2) parts[2 * cta + tid].rows = 0;
  if (st.bad && cta == 0 && tid == 0) raise_status(status, kStatusBadId);
  if (st.units == 0) return;
  __syncthreads();

  const uint32_t ring = smem_addr(smem) + warp * C::kStages * 2 * C::kTile;
  float* const jm = reinterpret_cast<float*>(smem + C::kRing);
  float* const jl = jm + kAWarps * kARows;
  float* const jo = jl + kAWarps * kARows;
  const float sc = a.scale * kLog2e;

  auto open = [&](WarpTile& t, int64_t left) {
    int fb;
    tile_blocks(plan, t.sq, t.tile, fb, t.nb);
    t.todo = static_cast<int>(min(static_cast<int64_t>(t.nb - t.blk), left));
    t.key0 = (fb + t.blk) * kABlock + warp * kWarpKeys;
    const int row0 = t.tile * kARows, end = min(row0 + kARows, t.sq.n * plan.group), before = t.sq.len - t.sq.n;
    t.lo = plan.window ? max(0, before + row0 / plan.group - plan.window + 1) : 0;
    t.hi = plan.causal ? min(t.sq.len, before + (end - 1) / plan.group + 1) : t.sq.len;
  };
  // Lane i: the page of step i0 + i of a tile, -1 where there is none.
  auto pages_of = [&](const WarpTile& t, int i0) {
    const int k = t.key0 + (i0 + lane) * kABlock;
    if (i0 + lane >= t.todo || k >= t.hi || k + kWarpKeys <= t.lo) return -1;
    const int id = b.table[static_cast<int64_t>(t.seq) * b.max_pages + (k >> c.page_shift)];
    if (id >= 0 && id < c.n_pages) return id;
    raise_status(status, kStatusBadId);
    return -1;
  };
  // Request this warp's keys and values of step i into ring slot `slot`; what
  // no row of the tile sees, or lies in no page, is not read and arrives as
  // zeros (a weight of zero would not silence a NaN there).
  auto request = [&](const WarpTile& t, int ids, int i, uint32_t slot) {
    const int k = t.key0 + i * kABlock;
    const int page = __shfl_sync(0xffffffffu, ids, i & 31);
    const int64_t off = static_cast<int64_t>(max(page, 0)) * c.page_stride + t.head * c.head_stride +
                        (k & (c.page_size - 1)) * c.slot_stride;
    const int first = t.lo - k, have = page < 0 ? 0 : t.hi - k;
    const uint32_t dst = ring + slot * 2 * C::kTile;
    constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll
    for (int n = 0; n < kWarpKeys * kChunks / 32; ++n) {
      const int p = n * 32 + lane, row = p / kChunks, ch = p % kChunks;
      const bool there = row >= first && row < have;
      const int64_t at = off + row * c.slot_stride + ch * 8;
      const uint32_t to = dst + row * D * 2 + ((ch ^ (row & 7)) << 4);
      cp_async16(to, there ? c.k + at : c.k, there);
      cp_async16(to + C::kTile, there ? c.v + at : c.v, there);
    }
  };

  WarpTile cur = {st.head, st.seq, st.tile, st.block, 0, 0, 0, 0, 0, st.sq}, nxt = cur;
  int64_t left = st.units, unit = st.first;  // unit: of cur's first block
  open(cur, left);
  int ids = pages_of(cur, 0), after = pages_of(cur, 32);  // of the 32 steps being requested, and of the 32 after them
  uint32_t base = 0;                                      // ring slot of cur's step 0
  auto slot_of = [&](int i) { return (base + static_cast<uint32_t>(i)) % C::kStages; };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (i < cur.todo) request(cur, ids, i, slot_of(i));
    cp_commit();
  }

  // A tile's queries: fragments of a 16 x D operand, rows past the end zero;
  // and the keys [lo, hi) that rows g and g + 8 see.
  uint32_t qf[D / 16][4];
  int lo[2], hi[2];
  auto load_queries = [&](const WarpTile& t) {
    const int row0 = t.tile * kARows, rows = t.sq.n * plan.group - row0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      const bool there = r < rows;
      const int tok = (row0 + r) / plan.group, qh = t.head * plan.group + (row0 + r) - tok * plan.group;
      const uint16_t* src = a.q + (t.sq.q0 + tok) * a.ldq + static_cast<int64_t>(qh) * D + 2 * qd;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][h] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * ks) : 0u;
        qf[ks][2 + h] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8) : 0u;
      }
      const int pos = t.sq.len - t.sq.n + tok;
      hi[h] = there ? (plan.causal ? min(t.sq.len, pos + 1) : t.sq.len) : 0;
      lo[h] = plan.window ? max(0, pos - plan.window + 1) : 0;
    }
  };
  load_queries(cur);

  for (bool first_seg = true;; first_seg = false) {
    // The next tile and its first pages are looked up now, and its first
    // steps requested behind cur's last: the copies go on while the warps are
    // joined (without this a CTA stood still for some 3 us per tile, of which
    // a batch of 64 sequences has 3.4 a CTA).
    const bool more = left > cur.todo + st.cost;
    int ids_n = -1;
    if (more) {
      nxt = cur;
      next_tile(plan, b, nxt.head, nxt.seq, nxt.tile, nxt.sq);
      nxt.blk = 0;
      open(nxt, left - cur.todo - st.cost);
      ids_n = pages_of(nxt, 0);
    }
    const bool flows = more && cur.todo >= kAhead && nxt.todo >= kAhead;

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    for (int i = 0; i < cur.todo; ++i) {
      const int ask = i + kAhead;
      if (ask < cur.todo) {
        if ((ask & 31) == 0) {
          ids = after;
          after = pages_of(cur, ask + 32);
        }
        request(cur, ids, ask, slot_of(ask));
      } else if (flows) {
        request(nxt, ids_n, ask - cur.todo, slot_of(ask));
      }
      cp_commit();
      cp_wait<kAhead>();
      __syncwarp();
      const int k = cur.key0 + i * kABlock;
      const uint32_t kt = ring + slot_of(i) * 2 * C::kTile, vt = kt + C::kTile;
      float s[2][4] = {};
      {
        // Matrices of a K load: keys 0-7 / 8-15 by elements 0-7 / 8-15 of the step.
        const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
          ldsm4(kt + row * D * 2 + (((2 * ks + half) ^ (row & 7)) << 4), f);
          mma16<T>(s[0], qf[ks], f[0], f[1]);
          mma16<T>(s[1], qf[ks], f[2], f[3]);
        }
      }
      uint32_t p[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = k + 8 * (j >> 1) + 2 * qd + (j & 1);
          x[j] = key >= lo[h] && key < hi[h] ? s[j >> 1][2 * h + (j & 1)] * sc : -INFINITY;
        }
        const float mx = quad_max(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
        const float mn = fmaxf(m[h], mx);
        const float base_m = mn == -INFINITY ? 0.0f : mn;  // no key seen yet: every weight below is exp2(-inf) = 0
        const float keep = exp2f(m[h] - base_m), top = base_m - kLift<T>;
        m[h] = mn;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = exp2f(x[j] - top);
        l[h] = l[h] * keep + ((x[0] + x[1]) + (x[2] + x[3]));
        // The weights enter the second product as 16-bit numbers (the type
        // the matrix instruction pairs with V's); the sum stays fp32.  A
        // second number for the rest of each would take as many instructions
        // again (200 sequences' step, fp16, d = 128: 90 us so, 99 with it).
        p[h] = pack2<T>(x[0], x[1]);
        p[2 + h] = pack2<T>(x[2], x[3]);
        if (__any_sync(0xffffffffu, keep != 1.0f)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * h] *= keep;
            o[n][2 * h + 1] *= keep;
          }
        }
      }
      {
        // Matrices of a (transposed) V load: keys 0-7 / 8-15 of elements
        // 0-7, then of elements 8-15.
        const int row = lane & 15, half = lane >> 4;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t f[4];
          ldsm4_t(vt + row * D * 2 + (((2 * n + half) ^ (row & 7)) << 4), f);
          mma16<T>(o[2 * n], p, f[0], f[1]);
          mma16<T>(o[2 * n + 1], p, f[2], f[3]);
        }
      }
      __syncwarp();  // the slot is refilled by the next step's copies
    }

    // Join the warps, eight rows at a time: every warp's m, l and O, then one
    // thread per four elements of a row, warps in order.
    const int row0 = cur.tile * kARows, rows = min(kARows, cur.sq.n * plan.group - row0);
    const bool whole = cur.blk == 0 && cur.todo == cur.nb;
    const int slot = first_seg ? 2 * cta : 2 * cta + 1;
    float* out = slots + slot * join_slot_floats(kARows, D);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (8 * h >= rows) break;
      const float lsum = quad_sum(l[h]);
      if (qd == 0) {
        jm[warp * kARows + 8 * h + g] = m[h];
        jl[warp * kARows + 8 * h + g] = lsum;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(jo + (warp * 8 + g) * D + 8 * n + 2 * qd) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
      __syncthreads();
      for (int e = tid; e < min(8, rows - 8 * h) * (D / 4); e += kAThreads) {
        const int rj = e / (D / 4), r = 8 * h + rj, col = (e % (D / 4)) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAWarps; ++w) mx = fmaxf(mx, jm[w * kARows + r]);
        const float base_m = mx == -INFINITY ? 0.0f : mx;
        float lt = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kAWarps; ++w) {
          const float f = exp2f(jm[w * kARows + r] - base_m);
          lt += f * jl[w * kARows + r];
          const float4 x = *reinterpret_cast<const float4*>(jo + (w * 8 + rj) * D + col);
          v.x += f * x.x;
          v.y += f * x.y;
          v.z += f * x.z;
          v.w += f * x.w;
        }
        // A row that sees nothing here is zero, whatever the values are that
        // other rows see (its weights of zero did not silence a NaN).
        if (lt == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (whole) {
          const float inv = lt > 0.0f ? 1.0f / lt : (lt == 0.0f ? 0.0f : lt);
          const int tok = (row0 + r) / plan.group, qh = cur.head * plan.group + (row0 + r) - tok * plan.group;
          store4<T>(a, cur.sq.q0 + tok, qh, D, col, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        } else {
          if (col == 0) {
            out[r] = mx;
            out[kARows + r] = lt;
          }
          *reinterpret_cast<float4*>(out + slot_o(kARows, r, col)) = v;
        }
      }
      __syncthreads();
    }
    if (!whole && cur.blk == 0 && tid == 0)
      parts[slot] = Part{cur.head, cur.sq.q0, row0, rows, share_of(st.work, st.used, unit + cur.nb - 1), {}};
    if (!more) break;
    left -= cur.todo + st.cost;
    unit += cur.todo + st.cost;
    base += cur.todo;
    cur = nxt;
    ids = ids_n;
    after = pages_of(cur, 32);
    load_queries(cur);
    if (!flows) {
      cp_wait<0>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i < cur.todo) request(cur, ids, i, slot_of(i));
        cp_commit();
      }
    }
  }
}

// Join the parts of the tiles that several CTAs did.  CTA (c, y) takes the
// tile whose first part CTA c of the attention kernel left (if any); the parts
// that follow are the first ones of CTAs c + 1 .. last.  Many rows or few parts (prompt
// chunks): a thread per piece of 4 columns.  Few rows in many parts (a decode
// step over a long cache has one tile in 40): the CTA's warps share the parts
// out, 32 pieces at a time, and their sums meet in shared memory.  Fixed
// order: the same sums every time.  Bound by latency: the parts are in L2; one
// sequence of 131 071 keys (40 parts a tile) adds 2 us to the call.
constexpr int kJoinWarps = 8;

struct RowSum {
  float m, l;
  float4 v;
  __device__ __forceinline__ void add(float mk, float lk, float4 x) {
    const float mn = fmaxf(m, mk), base = mn == -INFINITY ? 0.0f : mn;
    const float f0 = exp2f(m - base), f1 = exp2f(mk - base);
    m = mn;
    l = l * f0 + lk * f1;
    v.x = v.x * f0 + x.x * f1;
    v.y = v.y * f0 + x.y * f1;
    v.z = v.z * f0 + x.z * f1;
    v.w = v.w * f0 + x.w * f1;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    attn_join_kernel(const AttnArgs a, int slot_rows, const Divisor group, const Part* parts, const float* slots) {
  __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
  __shared__ float4 s_v[kJoinWarps][32];
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const Part p0 = parts[2 * c], p1 = parts[2 * c + 1];
  const bool second = p1.rows > 0;  // a CTA begins at most one tile that it does not end, its last
  const Part p = second ? p1 : p0;
  if (p.rows == 0) return;
  const size_t sf = join_slot_floats(slot_rows, D);
  const int lrow = (slot_rows + 3) & ~3, n = p.last - c + 1, items = p.rows * (D / 4);
  const float* s0 = slots + (2 * c + second) * sf;
  const bool many = n >= 4 && items <= static_cast<int>(64 * gridDim.y);
  const int step = many ? 32 : 32 * kJoinWarps;
  for (int base = blockIdx.y * step; base < items; base += gridDim.y * step) {
    const int e = base + (many ? lane : static_cast<int>(threadIdx.x));
    const bool there = e < items;
    const int r = there ? e % p.rows : 0, col = there ? (e / p.rows) * 4 : 0, at = slot_o(slot_rows, r, col);
    RowSum t = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll 4
    for (int k = many ? warp : 0; k < n; k += many ? kJoinWarps : 1) {
      const float* s = k == 0 ? s0 : slots + 2 * (c + k) * sf;
      t.add(s[r], s[lrow + r], *reinterpret_cast<const float4*>(s + at));
    }
    if (many) {
      __syncthreads();  // the sums of the pieces before have been read
      s_m[warp][lane] = t.m;
      s_l[warp][lane] = t.l;
      s_v[warp][lane] = t.v;
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) t.add(s_m[w][lane], s_l[w][lane], s_v[w][lane]);
    }
    if (!there) continue;
    const float inv = t.l > 0.0f ? 1.0f / t.l : (t.l == 0.0f ? 0.0f : t.l);  // a row that sees nothing is zero
    const int tok = (p.row0 + r) / group, qh = p.head * group + (p.row0 + r) - tok * group;
    store4<T>(a, p.q0 + tok, qh, D, col, make_float4(t.v.x * inv, t.v.y * inv, t.v.z * inv, t.v.w * inv));
  }
}

namespace {

// Which kernel a call takes, by the rows (tokens x query heads of a kv head)
// of an average sequence: kWarps for up to one 16-row tile, else the 128-row
// kernel, with two such tiles side by side where one does not hold them.
// Measured, 32 sequences of 2000 keys, 32/8 heads of 128 (of 64), us:
//   rows        4           16           20           128           136
//   kWarps      48 (30)     51 (32)      97 (58)      322 (173)     359 (191)
//   kTile       51 (37)     52 (38)      52 (38)      61 (40)       108 (72)
//   kTilePair   56 (48)     58 (49)      58 (49)      66 (51)       66 (51)
// These are sequences alike.  The host does not know their lengths, and an
// average says nothing of a long chunk among many short sequences: 255 steps
// of 2000 keys and 512 tokens on 8192 keys, 32/8 heads of 128, take 618 us in
// one call (kWarps) and 302 + 60 in two; 1000 tokens on 4000 keys 377 us with
// 255 sequences without new tokens, 60 without those.
enum Route { kWarps, kTile, kTilePair };
Route route(int64_t t, int64_t group, int64_t n_seqs) {
  const int64_t rows = (t * group + n_seqs - 1) / n_seqs;
  return rows <= kARows ? kWarps : rows <= (128 / group) * group ? kTile : kTilePair;
}
int attn_ctas() { return device_info().num_sms; }  // both kernels: one per SM
int route_rows(Route r, int group) { return r == kWarps ? kARows : attn_tile_rows(group, r == kTilePair); }

template <typename Kernel, typename... Args>
bool launch_pdl(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, args...));
}

template <typename T, int D>
int launch_warp(const KvCache& c, const KvBatch& b, const AttnArgs& a, int ctas, Part* parts, float* slots,
                unsigned* status, cudaStream_t s) {
  using C = WarpCfg<D>;
  const DeviceInfo& di = device_info();
  static std::atomic<bool> configured[64];  // per device (racing threads configure twice: idempotent)
  if (di.device < 0 || di.device >= 64) return TQ1_ERR_CUDA;
  if (!configured[di.device].load(std::memory_order_acquire)) {
    if (!cuda_ok(cudaFuncSetAttribute(attn_warp_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(C::kSmem))))
      return TQ1_ERR_CUDA;
    configured[di.device].store(true, std::memory_order_release);
  }
  const TilePlan plan = {Divisor(kARows), Divisor(a.n_q / c.n_kv), a.causal, a.window, kAShift};
  return launch_pdl(attn_warp_kernel<T, D>, dim3(ctas), kAThreads, C::kSmem, s, c, b, a, plan, parts, slots, status)
             ? TQ1_OK
             : TQ1_ERR_CUDA;
}

template <typename T, int D>
int launch_route(Route r, const KvCache& c, const KvBatch& b, const AttnArgs& a, void* ws, unsigned* status,
                 cudaStream_t s) {
  const int ctas = attn_ctas(), group = a.n_q / c.n_kv;
  Part* parts = static_cast<Part*>(ws);
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + join_parts_bytes(ctas));
  int rc = TQ1_ERR_UNSUPPORTED;
  if (r != kWarps) rc = launch_attn_tile(c, b, a, r == kTilePair, ctas, parts, slots, status, s);
  if (rc == TQ1_ERR_UNSUPPORTED) {  // or strides that a tensor map cannot describe
    r = kWarps;
    rc = launch_warp<T, D>(c, b, a, ctas, parts, slots, status, s);
  }
  if (rc != TQ1_OK) return rc;
  const int rows = route_rows(r, group);
  // CTAs that share out a tile's rows.  Of 16 rows: one short sequence 7.8 us
  // with 8, 8.3 with 16.  Of 128 and more, us with 8 / 12 / 16 / 32: three
  // small chunks 18.9 / 17.2 / 16.7 / 17.1, ragged mix 45.5 / 45.4 / 45.8 / 46.8.
  const int share = std::min(r == kWarps ? 8 : 12, (rows * (D / 4) + 31) / 32);
  return launch_pdl(attn_join_kernel<T, D>, dim3(ctas, share), 32 * kJoinWarps, 0, s, a, rows, Divisor(group),
                    static_cast<const Part*>(parts), static_cast<const float*>(slots))
             ? TQ1_OK
             : TQ1_ERR_CUDA;
}

}  // namespace

// What a call of exactly these sizes needs: fewer bytes where more sequences
// share the tokens (64 tokens, group 4, d = 128: 2.5 MB of 64 sequences, 40 MB
// of one).
size_t attn_workspace_bytes(const KvCache& c, int64_t t, int64_t n_q, int64_t n_seqs) {
  const int group = static_cast<int>(n_q / c.n_kv);
  if (group < 1 || group > 128) return 0;
  const int ctas = attn_ctas(), rows = std::max(kARows, route_rows(route(t, group, n_seqs), group));
  const size_t b = join_parts_bytes(ctas) + 2 * static_cast<size_t>(ctas) * join_slot_floats(rows, c.d) * sizeof(float);
  return (b + 255) & ~size_t(255);
}

int launch_attn(const KvCache& c, const KvBatch& b, const AttnArgs& a, void* ws, unsigned* status, cudaStream_t s) {
  const Route r = route(b.t, a.n_q / c.n_kv, b.n_seqs);
  if (c.d == 128)
    return c.dtype == kBf16 ? launch_route<__nv_bfloat16, 128>(r, c, b, a, ws, status, s)
                            : launch_route<__half, 128>(r, c, b, a, ws, status, s);
  return c.dtype == kBf16 ? launch_route<__nv_bfloat16, 64>(r, c, b, a, ws, status, s)
                          : launch_route<__half, 64>(r, c, b, a, ws, status, s);
}

}  // namespace tq1
