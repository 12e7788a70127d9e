// rope.cu -- rotary positions, and the append of rotated keys and of values
// to the paged cache.
//
// A head's first `rot` elements are rot/2 pairs; pair i of the token at
// position p turns by the angle a = p * f_i (f: inv_freq):
//   x' = m (x cos a - y sin a),   y' = m (x sin a + y cos a)
// with (x, y) = elements (i, i + rot/2), or (2i, 2i + 1) when interleaved;
// the head's other elements are copied.  q goes to q_out, k and v to the slot
// that the token's position in its sequence names, so a projection's output
// is read once and every result written once.
//
// The angle: p f_i reaches 10^5 and more radians, where an fp32 product is
// already off by 0.01.  It is formed in fp64, in half turns, and reduced
// there; the rest, below one half turn, goes to sincospif.  Four fp64
// operations per angle, and one angle serves all heads of a token.
//
// Bound: HBM for chunks (6 bytes per value in, out); latency for a step.
// A thread does 8 elements of one head: two 4-element halves of the "half"
// layout (4 pairs), or 8 neighbours, so that a warp's accesses are whole
// 128-byte lines (16-byte loads, 8- or 16-byte stores).
#include "../../include/tq1.h"
#include "kv.cuh"
#include "tq1_internal.h"

namespace tq1 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRotPairs = 128;  // head_dim <= 256
constexpr int kPer = 2;            // tokens of a CTA, where there are many
constexpr int kRopeCtas = 6;       // CTAs an SM holds (40 registers a thread): what hides the loads

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]) {
  const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
  const float2 a = unpack2<T>(x.x), b = unpack2<T>(x.y);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

// One CTA: `per` tokens from blockIdx.x * per on, and of each token's heads
// (of q, k and v) the blockIdx.y-th part of gridDim.y.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_append_kernel(const KvCache c, const KvBatch b, const RopeArgs a, int per, int one_wave, unsigned* status) {
  __shared__ float2 s_cs[kPer][kMaxRotPairs];
  __shared__ int s_seq[kPer], s_pos[kPer], s_page[kPer];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tok0 = blockIdx.x * per;
  // A thread keeps its group of 8 elements and walks the CTA's (token, head)
  // pairs with a step and a compare.  One pair at a time and two tokens a
  // CTA: what hides the loads is many resident threads, not many loads each
  // (12 381 tokens of 40 + 2 x 8 heads of 128: 86 us, 6.2 TB/s; with two or
  // four pairs held per thread 97 and 106 us, with four or eight tokens a CTA
  // 90 and 92 us).
  const int pairs = a.rot >> 1, groups = c.d >> 3, heads = a.n_q + 2 * c.n_kv;
  const int h_lo = static_cast<int>(static_cast<int64_t>(heads) * blockIdx.y / gridDim.y);
  const int h_n = static_cast<int>(static_cast<int64_t>(heads) * (blockIdx.y + 1) / gridDim.y) - h_lo;
  const int stride = kRopeThreads / groups, grp = tid % groups;
  const bool in_rot = grp < (a.rot >> 3), halves = in_rot && !a.interleaved;
  // Elements e0 .. e0+3 and e1 .. e1+3 of the head; of v always 8 neighbours.
  const int n0 = 8 * grp, n1 = n0 + 4, e0 = halves ? 4 * grp : n0, e1 = halves ? e0 + pairs : n1;
  const int upto = tid < stride * groups ? min(per, b.t - tok0) : 0;  // tokens; threads past the last whole head idle
  int w = 0, h = tid / groups;
  auto settle = [&]() {
    while (w < upto && h >= h_n) {
      h -= h_n;
      ++w;
    }
  };
  settle();
  float x[4], y[4];
  int u = -1, head = 0;  // token and head of what x and y hold; token -1: nothing left
  auto fetch = [&]() {
    u = w < upto ? w : -1;
    head = h_lo + h;
    if (u < 0) return;
    const bool is_q = head < a.n_q, is_v = head >= a.n_q + c.n_kv, turn = in_rot && !is_v;
    const TI* src = static_cast<const TI*>(is_q ? a.q : is_v ? a.v : a.k) +
                    static_cast<int64_t>(tok0 + u) * (is_q ? a.ldq : is_v ? a.ldv : a.ldk) +
                    static_cast<int64_t>(is_q ? head : is_v ? head - a.n_q - c.n_kv : head - a.n_q) * c.d;
    load4(src + (turn ? e0 : n0), x);
    load4(src + (turn ? e1 : n1), y);
    h += stride;
    settle();
  };
  if (one_wave) pdl_launch_dependents();
  pdl_wait();
  fetch();  // on their way while the tokens' places are looked up
  // One angle per thread: pair ap of token at.
  static_assert(kPer == 2 && kPer * kMaxRotPairs <= kRopeThreads, "an angle per thread");
  const int at = tid >= pairs, ap = tid - at * pairs;
  const bool angle = tid < per * pairs && tok0 + at < b.t;
  const float freq = angle ? a.inv_freq[ap] : 0.0f;
  // The sequence of each token, its position and its page: a warp per token.
  if (warp < per) {
    const int tok = tok0 + warp;
    int seq = -1, pos = 0, page = -1;
    if (tok < b.t) {
      int count = 0;  // sequences that end at or before this token
      for (int s = lane; s < b.n_seqs; s += 32) count += b.q_start[s + 1] <= tok;
      count = __reduce_add_sync(0xffffffffu, count);
      int begin = b.t, end = 0, len = 0;  // of the sequence, read at once
      if (count < b.n_seqs) {
        begin = b.q_start[count];
        end = b.q_start[count + 1];
        len = b.kv_len[count];
      }
      if (begin <= tok) {
        seq = count;
        pos = len - (end - tok);
        if (pos >= 0 && pos < b.max_len) {
          page = b.table[static_cast<int64_t>(seq) * b.max_pages + (pos >> c.page_shift)];
          if (page < 0 || page >= c.n_pages) page = -1;
        }
        if (page < 0 && lane == 0 && blockIdx.y == 0) raise_status(status, kStatusBadId);
      }
    }
    if (lane == 0) {
      s_seq[warp] = seq;
      s_pos[warp] = pos;
      s_page[warp] = page;
    }
  }
  __syncthreads();
  if (angle && s_seq[at] >= 0) {
    const int pos = a.positions ? a.positions[tok0 + at] : s_pos[at];
    double half_turns = static_cast<double>(pos) * static_cast<double>(freq) * 0.31830988618379067154;
    half_turns -= 2.0 * rint(0.5 * half_turns);
    float sn, cs;
    sincospif(static_cast<float>(half_turns), &sn, &cs);
    s_cs[at][ap] = make_float2(cs * a.mscale, sn * a.mscale);
  }
  __syncthreads();
  for (; u >= 0; fetch()) {
    const bool is_q = head < a.n_q, is_v = head >= a.n_q + c.n_kv, turn = in_rot && !is_v;
    if (s_seq[u] < 0 || (!is_q && s_page[u] < 0)) continue;
    TO* dst;
    if (is_q)
      dst = reinterpret_cast<TO*>(a.q_out) + (static_cast<int64_t>(tok0 + u) * a.n_q + head) * c.d;
    else
      dst = reinterpret_cast<TO*>(is_v ? c.v : c.k) + s_page[u] * c.page_stride +
            (is_v ? head - a.n_q - c.n_kv : head - a.n_q) * c.head_stride + (s_pos[u] & (c.page_size - 1)) * c.slot_stride;
    const float2* cs = s_cs[u];
    if (turn && halves) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = cs[e0 + j];
        const float v = x[j] * t.x - y[j] * t.y;
        y[j] = x[j] * t.y + y[j] * t.x;
        x[j] = v;
      }
    } else if (turn) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 t0 = cs[(e0 >> 1) + j], t1 = cs[(e1 >> 1) + j];
        float v = x[2 * j] * t0.x - x[2 * j + 1] * t0.y;
        x[2 * j + 1] = x[2 * j] * t0.y + x[2 * j + 1] * t0.x;
        x[2 * j] = v;
        v = y[2 * j] * t1.x - y[2 * j + 1] * t1.y;
        y[2 * j + 1] = y[2 * j] * t1.y + y[2 * j + 1] * t1.x;
        y[2 * j] = v;
      }
    }
    const uint2 lo = make_uint2(pack2<TO>(x[0], x[1]), pack2<TO>(x[2], x[3]));
    const uint2 hi = make_uint2(pack2<TO>(y[0], y[1]), pack2<TO>(y[2], y[3]));
    if (turn && halves) {
      *reinterpret_cast<uint2*>(dst + e0) = lo;
      *reinterpret_cast<uint2*>(dst + e1) = hi;
    } else {
      *reinterpret_cast<uint4*>(dst + n0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

// f_i = theta_i ((1 - g) / factor + g), theta_i = base^(-2i / rot), where g
// ramps from 0 to 1 with the turns orig_len theta_i / 2 pi that the pair makes
// over the original context, between `low` and `high` turns: fast pairs keep
// their frequency, slow ones are stretched by the factor.  fp64, rounded once.
__global__ void rope_freqs_kernel(float* inv_freq, int pairs, double base, double factor, double orig_len, double low,
                                  double high) {
  pdl_wait();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const double theta = pow(base, -static_cast<double>(i) / pairs);
    double g = 1.0;
    if (factor != 1.0) {
      const double turns = orig_len * theta * 0.15915494309189533577;
      g = high > low ? (turns - low) / (high - low) : (turns >= high ? 1.0 : 0.0);
      g = fmin(fmax(g, 0.0), 1.0);
    }
    inv_freq[i] = static_cast<float>(theta * ((1.0 - g) / factor + g));
  }
}

template <typename TI, typename TO>
int launch(const KvCache& c, const KvBatch& b, const RopeArgs& a, unsigned* status, cudaStream_t s) {
  // Two tokens a CTA share its start; while that leaves SMs without a CTA,
  // one token a CTA, its heads split over as many CTAs as leave a thread one
  // group of 8 elements.
  const int items = (a.n_q + 2 * c.n_kv) * (c.d >> 3);
  const int sms = device_info().num_sms;
  const int per = b.t >= 8 * sms ? kPer : 1;
  const int64_t gx = (static_cast<int64_t>(b.t) + per - 1) / per;
  int gy = 1;
  while (gy < 16 && gx * gy < 2 * sms && items > gy * kRopeThreads) ++gy;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, rope_append_kernel<TI, TO>, c, b, a, per, gx * gy <= 2 * sms ? 1 : 0, status)) ? TQ1_OK : TQ1_ERR_CUDA;
}

template <typename TO>
int launch_out(const KvCache& c, const KvBatch& b, const RopeArgs& a, unsigned* status, cudaStream_t s) {
  switch (a.in_dtype) {
    case kF16: return launch<__half, TO>(c, b, a, status, s);
    case kBf16: return launch<__nv_bfloat16, TO>(c, b, a, status, s);
    default: return launch<float, TO>(c, b, a, status, s);
  }
}

}  // namespace

int launch_rope_append(const KvCache& c, const KvBatch& b, const RopeArgs& a, unsigned* status, cudaStream_t s) {
  return c.dtype == kBf16 ? launch_out<__nv_bfloat16>(c, b, a, status, s) : launch_out<__half>(c, b, a, status, s);
}

int launch_rope_freqs(float* inv_freq, int rot, double base, double factor, double orig_len, double low, double high,
                      cudaStream_t s) {
  rope_freqs_kernel<<<1, 128, 0, s>>>(inv_freq, rot / 2, base, factor, orig_len, low, high);
  return cuda_ok(cudaGetLastError()) ? TQ1_OK : TQ1_ERR_CUDA;
}

}  // namespace tq1
