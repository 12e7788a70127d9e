// kv.cuh -- the paged key/value cache as the kernels see it, 16-bit element
// helpers, and the division of an attention call's work among its CTAs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_internal.h"
#include "tq1_device.cuh"

namespace tq1 {

// ------------------------------------------------------ 16-bit elements --
// Two fp32 values to two 16-bit elements (round to nearest), the first in the
// low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// --------------------------------------------------------- the sequences --
// New tokens [q0, q0 + n) and cache length of one sequence.  The arrays are
// device data the host has not seen, so they are clamped to what exists: no
// index formed from them leaves the call's tensors.  The kernels here begin
// while the one before them may still write what they read after their wait,
// so none of it goes through read-only loads (__ldg), which take data that
// does not change while a kernel runs and may be moved ahead of the wait.
struct Seq {
  int q0, n, len;
};
__device__ __forceinline__ Seq load_seq(const KvBatch& b, int s) {
  Seq r;
  int q0 = b.q_start[s], q1 = b.q_start[s + 1];
  r.len = min(max(b.kv_len[s], 0), b.max_len);
  q0 = min(max(q0, 0), b.t);
  q1 = min(max(q1, q0), b.t);
  r.q0 = q0;
  r.n = q1 - q0;
  return r;
}

// ------------------------------------------------- division of attention --
// The (token, query head of the group) pairs of one sequence and one kv head
// are its rows, row = token * group + head, cut into tiles of `rows` rows.
// A tile reads the cache in blocks of `block` keys, from the first key any
// of its rows sees to the last.  The call's work is the list of (kv head,
// sequence, tile, block), in that order, where a tile's blocks come after
// `cost` units for its beginning and end; CTA c of C does the units
// [W c / C, W (c+1) / C) of the W in the list.  So every CTA has the same
// work to one unit whatever the sequences' lengths are, and only the tiles at
// a CTA's two ends are shared: their parts are joined afterwards.  (A share
// that ends within a tile's cost does nothing of the tile, and one that begins
// there begins with its first block.)
struct TilePlan {
  Divisor rows, group;
  int causal, window;
  int shift;  // log2 of a block's keys
};

// What a tile costs beside its blocks, in blocks: its queries, the first
// block's latency, the last product, its output (2 us of the tensor-core
// kernel).  Without it a CTA with six tiles was done 6 us after one with three
// (ragged mix of 1 to 1463 tokens, us with 0 / 1 / 2 / 3 / 4 / 6: 53.2 / 48.9 /
// 48.5 / 47.5 / 47.3 / 48.2; decode step of 64 sequences: 153 / 148 / 146 /
// 145 / 146 / 151; 12 sequences of up to 1500 tokens and 5000 keys, 24/8 heads
// of 128: 167 / 156 / 150 / 146 / 148 / 151).  Shares of so few blocks that
// a tile's cost is most of them want one less (decode step of 8 sequences of
// 200 to 900 keys, us with 0 / 1 / 2 / 3: 11.8 / 11.5 / 10.6 / 10.9; three
// chunks of 30 to 90 tokens: 20.0 / 19.9 / 19.9 / 21.2).
constexpr int kTileCost = 3;

// Blocks of one tile: the first one and how many.  A tile whose rows see
// nothing has one block (it is masked whole; its rows come out as zeros).
__device__ __forceinline__ void tile_blocks(const TilePlan& p, const Seq& s, int tile, int& first, int& count) {
  const int r0 = tile * p.rows, r1 = min(r0 + p.rows, s.n * p.group);
  const int tok0 = r0 / p.group, tok1 = (r1 - 1) / p.group;
  const int pos0 = s.len - s.n + tok0, pos1 = s.len - s.n + tok1;
  const int hi = p.causal ? min(s.len, pos1 + 1) : s.len;
  const int lo = p.window ? max(0, pos0 - p.window + 1) : 0;
  first = lo >> p.shift;
  count = max(1, ((hi + (1 << p.shift) - 1) >> p.shift) - first);
  if (hi <= lo) count = 1;
}
__device__ __forceinline__ int seq_tiles(const TilePlan& p, const Seq& s) {
  return (s.n * p.group + p.rows - 1) / p.rows;
}

// Inclusive sum over a warp's lanes.
template <typename I>
__device__ __forceinline__ I warp_scan(I v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// Inclusive sum over the block's threads in thread order; `s_warp` holds one
// int per warp.  Returns the inclusive sum, and the block's total in `total`.
template <int NT>
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  __syncthreads();  // s_warp may still be read from the call before
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int x = s_warp[w];
    if (w < warp) before += x;
    total += x;
  }
  return v + before;
}

// Where CTA `cta` of `ctas` begins and how much it does.
struct Start {
  int head, seq, tile, block;  // first unit
  int64_t first, units;        // its place in the list, units of this CTA from there on (0: none)
  int64_t work;                // units of the call
  int used;                    // CTAs that have some
  int cost;                    // units of a tile beside its blocks
  bool bad;                    // starts that do not ascend: there is no work
  Seq sq;                      // of `seq`
};

// Unit u0 of share c of `work` units over `used` shares, and the share that
// has unit u.
__device__ __forceinline__ int64_t share_begin(int64_t work, int used, int c) {
  if (work < (int64_t{1} << 31)) {  // 32-bit divisions: a 64-bit one takes some hundred instructions
    const uint32_t q = static_cast<uint32_t>(work) / static_cast<uint32_t>(used), r = static_cast<uint32_t>(work) - q * used;
    return static_cast<int64_t>(q) * c + min(static_cast<uint32_t>(c), r);
  }
  const int64_t q = work / used, r = work - q * used;
  return q * c + min(static_cast<int64_t>(c), r);
}
__device__ __forceinline__ int share_of(int64_t work, int used, int64_t u) {
  const int64_t q = work / used, r = work - q * used, longer = (q + 1) * r;
  return static_cast<int>(u < longer ? u / (q + 1) : r + (u - longer) / q);
}

// Called by all NT threads; every warp has the result.  `s_nb`: at least 12
// n_seqs bytes of shared memory, still read by other warps when the call
// returns.  One barrier: the search stands before anything else of the call,
// and of a small call it was the larger part (a form with a block-wide sum per
// step took 5 us of the 70 us of a ragged batch of prompt chunks).
template <int NT>
__device__ __forceinline__ Start find_start(const TilePlan& p, const KvBatch& b, int n_kv, int cta, int ctas, int64_t* s_nb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* const s_nt = reinterpret_cast<int*>(s_nb + b.n_seqs);
  // Sequences that share no token have at most this many tiles (2^26 + 2^13).
  // Starts that do not ascend can make them share tokens, up to n_seqs times
  // as many; all the counts below rely on this limit, so such a call is
  // refused, and no warp counts the blocks of more tiles than that.
  const int most = b.t * p.group / p.rows + b.n_seqs;
  int counted = 0;
  // Blocks and tiles of each sequence: by its thread where it has one tile, else (left
  // as -1) by a warp, a lane per tile.
  for (int s0 = 32 * warp; s0 < b.n_seqs; s0 += NT) {
    const int s = s0 + lane;
    int nb = 0;
    if (s < b.n_seqs) {
      const Seq q = load_seq(b, s);
      const int tiles = seq_tiles(p, q);
      int f;
      if (tiles == 1) tile_blocks(p, q, 0, f, nb);
      if (tiles > 1) nb = -1;
      s_nb[s] = nb;
      s_nt[s] = tiles;
    }
    __syncwarp();
    for (uint32_t more = __ballot_sync(0xffffffffu, nb < 0); more; more &= more - 1) {
      const int t = s0 + __ffs(more) - 1;
      const Seq q = load_seq(b, t);
      const int tiles = seq_tiles(p, q);
      int64_t sum = 0;
      counted = min(counted + tiles, most + 1);
      for (int i = lane; i < tiles && counted <= most; i += 32) {
        int f, c;
        tile_blocks(p, q, i, f, c);
        sum += c;
      }
      sum = warp_scan(sum);
      if (lane == 31) s_nb[t] = sum;
    }
  }
  __syncthreads();
  // A lane per run of sequences: their sum, the sum of all, and the lane
  // whose run holds the first unit.
  const int run = (b.n_seqs + 31) >> 5, s0 = lane * run, s1 = min(s0 + run, b.n_seqs);
  int64_t mine = 0, many = 0;
  for (int s = s0; s < s1; ++s) {
    mine += s_nb[s];
    many += s_nt[s];
  }
  int64_t end = warp_scan(mine);
  const uint32_t mine_t = static_cast<uint32_t>(min(many, int64_t{most} + 1));
  const uint32_t end_t = warp_scan(mine_t), all_t = __shfl_sync(0xffffffffu, end_t, 31);  // 32 (most + 1) < 2^32
  int64_t all = __shfl_sync(0xffffffffu, end, 31);  // blocks of one kv head
  Start r;
  r.bad = all_t > static_cast<uint32_t>(most);
  r.cost = !r.bad && all * n_kv < static_cast<int64_t>(kTileCost) * ctas ? kTileCost - 1 : kTileCost;
  mine += static_cast<int64_t>(r.cost) * mine_t;
  end += static_cast<int64_t>(r.cost) * end_t;
  all += static_cast<int64_t>(r.cost) * all_t;  // units of one kv head
  const int64_t work = r.bad ? 0 : all * n_kv;
  const int used = static_cast<int>(min(work, static_cast<int64_t>(ctas)));  // fewer units than CTAs: one each
  r.work = work;
  r.used = used;
  r.first = 0;
  r.units = 0;
  r.head = r.seq = r.tile = r.block = 0;
  r.sq = Seq{0, 0, 0};
  if (cta >= used) return r;
  r.first = share_begin(work, used, cta);
  r.units = share_begin(work, used, cta + 1) - r.first;
  r.head = work < (int64_t{1} << 31) ? static_cast<uint32_t>(r.first) / static_cast<uint32_t>(all) : static_cast<int>(r.first / all);
  int64_t rem = r.first - r.head * all;
  const int owner = __ffs(__ballot_sync(0xffffffffu, rem < end)) - 1;
  int seq = s0;
  int64_t into = rem - (end - mine);
  if (lane == owner)
    for (int64_t u; into >= (u = s_nb[seq] + static_cast<int64_t>(r.cost) * s_nt[seq]); ++seq) into -= u;
  r.seq = __shfl_sync(0xffffffffu, seq, owner);
  rem = __shfl_sync(0xffffffffu, into, owner);
  const Seq q = load_seq(b, r.seq);
  r.sq = q;
  const int tiles = seq_tiles(p, q);
  r.block = static_cast<int>(rem);
  for (int base = 0; tiles > 1 && base < tiles; base += 32) {
    int f, c = 0;
    if (base + lane < tiles) {
      tile_blocks(p, q, base + lane, f, c);
      c += r.cost;
    }
    const int upto = warp_scan(c), sum = __shfl_sync(0xffffffffu, upto, 31);
    if (rem < sum) {
      const int hit = __ffs(__ballot_sync(0xffffffffu, rem < upto)) - 1;
      r.tile = base + hit;
      r.block = static_cast<int>(rem) - __shfl_sync(0xffffffffu, upto - c, hit);
      break;
    }
    rem -= sum;
  }
  // From the tile's units to its blocks.
  const int rest = max(r.cost - r.block, 0);
  r.block = max(r.block - r.cost, 0);
  r.first += rest;
  r.units = max(r.units - rest, int64_t{0});
  return r;
}

// The next tile after (head, seq, tile); there is one, since the CTA has
// units left.
__device__ __forceinline__ void next_tile(const TilePlan& p, const KvBatch& b, int& head, int& seq, int& tile, Seq& q) {
  if (++tile < seq_tiles(p, q)) return;
  tile = 0;
  for (int i = 0; i <= b.n_seqs; ++i) {  // at most once around: sequences without new tokens have no tiles
    if (++seq == b.n_seqs) {
      seq = 0;
      ++head;
    }
    q = load_seq(b, seq);
    if (q.n > 0) return;
  }
}

// ------------------------------------------------------------ the joining --
// What a CTA left of a tile it did not do alone (its first or its last):
// rows of m, l and unnormalised O in the workspace, described by a Part.
struct Part {
  int head, q0, row0;  // kv head, first token of the sequence, first row of the tile
  int rows;            // rows, in the part with the tile's first block; 0 in the others and where there is none
  int last;            // the CTA that has the tile's last block
  int pad[3];
};

// Workspace of `ctas` CTAs: their parts, then two slots each of rows * (d + 2)
// floats: m [rows] (in log2 units), l [rows], then O four columns at a time,
// [d/4][rows][4], so that threads of consecutive rows store consecutive
// 16-byte pieces.
inline __host__ __device__ size_t join_parts_bytes(int ctas) { return static_cast<size_t>(ctas) * 2 * sizeof(Part); }
inline __host__ __device__ size_t join_slot_floats(int rows, int d) { return static_cast<size_t>((rows + 3) & ~3) * (d + 2); }
__device__ __forceinline__ int slot_o(int rows, int r, int col) { return 2 * ((rows + 3) & ~3) + col * rows + 4 * r; }

constexpr float kLog2e = 1.4426950408889634f;

// Store elements e .. e+3 of an output row.
template <typename T>
__device__ __forceinline__ void store4(const AttnArgs& a, int64_t tok, int head, int d, int e, float4 v) {
  const int64_t at = tok * a.ldo + static_cast<int64_t>(head) * d + e;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
}

}  // namespace tq1
