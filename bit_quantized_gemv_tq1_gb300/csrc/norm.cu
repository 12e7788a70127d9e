// norm.cu -- the residual's addition, the root-mean-square norm and the
// Q8_1 rows that the next product takes, in one pass:
//   x' = x + delta,   y = gamma x' / sqrt(mean(x'^2) + eps),   Q8_1(y)
// with the quantiser's operations (d = max|y| / 127, q = round half away
// (y / d)), so that the blocks equal q8_1_quantize_acts of y bit for bit.
//
// One CTA a row.  A thread holds NV groups of eight values in registers
// between the sum of squares and the scaling (NV = 0: rows too long for that
// are read again), four neighbouring lanes hold a Q8_1 block: two shuffles
// give its maximum and its sum.  Sums of squares are fp32, a thread's in order,
// then by shuffles: the same bits in every call of as many rows.  How many groups a
// thread has goes by the number of rows, so a row may have other last bits in a batch
// of another size.  (The same order whatever the batch, spans of 32 groups at a time,
// took 2 to 4% more of many rows without a delta.)
//
// A few rows wait for their loads, then for the row's sum: a row of 6144 takes
// 2.7 us in a sequence of calls, 48 rows of 5120 with an fp32 delta 3.2.  Many
// are bound by memory: 4096 rows of 5120 with a bf16 delta in 41.4 us, 5.6 TB/s.
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

struct NoDelta {};
template <typename TD>
constexpr uint32_t delta_size() {
  return std::is_same<TD, NoDelta>::value ? 0 : static_cast<uint32_t>(sizeof(TD));
}

constexpr int kSlots = 2;                  // rows on their way, or being read
constexpr int64_t kRowsSmem = 200 * 1024;
constexpr int kRowsMinK = 6144;

// Eight values; x' = x + delta of a group.
struct Eight {
  float4 a, b;
};
__device__ __forceinline__ float4 add4(const float4& x, const float4& y) {
  return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}
__device__ __forceinline__ Eight load8(const float* p, int i) {
  const float4* q = reinterpret_cast<const float4*>(p) + 2 * i;
  return {q[0], q[1]};
}
template <typename T>
__device__ __forceinline__ Eight load8(const T* p, int i) {
  const uint4 x = reinterpret_cast<const uint4*>(p)[i];
  const float2 a = unpack2<T>(x.x), b = unpack2<T>(x.y), c = unpack2<T>(x.z), d = unpack2<T>(x.w);
  return {make_float4(a.x, a.y, b.x, b.y), make_float4(c.x, c.y, d.x, d.y)};
}

// A row's parts of the call's tensors.
struct RowOf {
  const float* x;
  const void* delta;
  const float* gamma;
  float* x_out;
  uint32_t* q8;
  void* y;
  int y_type;
};

template <typename TD>
__device__ __forceinline__ RowOf row_of(const NormArgs& a, int64_t row) {
  const int64_t at = row * a.k;
  RowOf r;
  r.x = a.x + at;
  if constexpr (!std::is_same<TD, NoDelta>::value) r.delta = static_cast<const TD*>(a.delta) + at;
  r.gamma = a.gamma;
  r.x_out = a.x_out ? a.x_out + at : nullptr;
  r.q8 = a.q8 ? a.q8 + row * (a.k >> 5) * 9 : nullptr;
  r.y = a.y ? static_cast<uint8_t*>(a.y) + at * (a.y_type == kF32 ? 4 : 2) : nullptr;
  r.y_type = a.y_type;
  return r;
}

template <typename TD>
__device__ __forceinline__ Eight load_x(const RowOf& r, int i) {
  Eight v = load8(r.x, i);
  if constexpr (!std::is_same<TD, NoDelta>::value) {
    const Eight d = load8(static_cast<const TD*>(r.delta), i);
    v = {add4(v.a, d.a), add4(v.b, d.b)};
  }
  return v;
}
__device__ __forceinline__ void store_x(const RowOf& r, int i, const Eight& v) {
  float4* q = reinterpret_cast<float4*>(r.x_out) + 2 * i;
  q[0] = v.a;
  q[1] = v.b;
}

__device__ __forceinline__ float square_sum(const Eight& v, float s) {
  s = fmaf(v.a.x, v.a.x, fmaf(v.a.y, v.a.y, fmaf(v.a.z, v.a.z, fmaf(v.a.w, v.a.w, s))));
  return fmaf(v.b.x, v.b.x, fmaf(v.b.y, v.b.y, fmaf(v.b.z, v.b.z, fmaf(v.b.w, v.b.w, s))));
}

// The quantiser's rounding of one value: q8_1_quantize_acts' operations.
__device__ __forceinline__ uint32_t round8(float v, float d) {
  const float r = roundf(__fdiv_rn(v, d));
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(r, -127.0f), 127.0f)));
}

// The same of four values, packed: v / d is within 2e-5 of v * (1 / d) (two
// roundings of numbers up to 127), so the nearest integer is the quantiser's
// but where that lies within 3e-5 of a half; there (one value in 8000) the
// quotient is formed, and where values are not finite.  The integer is read off
// the last bits of 1.5 2^23 + v/d.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ uint32_t round8x4(const float4& v, float d, float inv) {
  constexpr float kMagic = 12582912.0f;
  const float t[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  float off = 0.0f;
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float m = __fadd_rn(t[i], kMagic);
    q[i] = __float_as_uint(m);
    off = max_or_nan(off, fabsf(t[i] - __fsub_rn(m, kMagic)));
  }
  if (!(off <= 0.49997f) || !(d > 1e-36f)) {  // 1 / d of smaller ones is not finite
    q[0] = round8(v.x, d);
    q[1] = round8(v.y, d);
    q[2] = round8(v.z, d);
    q[3] = round8(v.w, d);
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

__device__ __forceinline__ float4 scaled(const float4& v, float inv, const float4& g) {
  return make_float4(__fmul_rn(__fmul_rn(v.x, inv), g.x), __fmul_rn(__fmul_rn(v.y, inv), g.y), __fmul_rn(__fmul_rn(v.z, inv), g.z),
                     __fmul_rn(__fmul_rn(v.w, inv), g.w));
}
__device__ __forceinline__ float most(const float4& v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const Eight& v) {
  return make_uint4(pack2<T>(v.a.x, v.a.y), pack2<T>(v.a.z, v.a.w), pack2<T>(v.b.x, v.b.y), pack2<T>(v.b.z, v.b.w));
}

// Scales group i of the row, writes y and the group's two words of its Q8_1
// block.  Every lane of the warp calls this; the four lanes of a block are live together.
__device__ __forceinline__ void finish(const RowOf& r, int i, bool live, Eight v, float inv) {
  if (live) {
    Eight g = {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(1.f, 1.f, 1.f, 1.f)};
    if (r.gamma) g = load8(r.gamma, i);
    v = {scaled(v.a, inv, g.a), scaled(v.b, inv, g.b)};
    if (r.y) {
      if (r.y_type == kF32) {
        static_cast<float4*>(r.y)[2 * i] = v.a;
        static_cast<float4*>(r.y)[2 * i + 1] = v.b;
      } else {
        static_cast<uint4*>(r.y)[i] = r.y_type == kF16 ? pack8<__half>(v) : pack8<__nv_bfloat16>(v);
      }
    }
  }
  if (!r.q8) return;
  float m = fmaxf(most(v.a), most(v.b));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float d = __fdiv_rn(m, 127.0f);
  uint32_t lo = 0, hi = 0;
  if (live && d != 0.0f) {
    const float over = __frcp_rn(d);
    lo = round8x4(v.a, d, over);
    hi = round8x4(v.b, d, over);
  }
  int sum = __dp4a(static_cast<int>(hi), 0x01010101, __dp4a(static_cast<int>(lo), 0x01010101, 0));
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  if (!live) return;
  uint32_t* blk = r.q8 + (i >> 2) * 9;
  blk[1 + 2 * (i & 3)] = lo;
  blk[2 + 2 * (i & 3)] = hi;
  if ((i & 3) == 0) {
    const uint32_t d16 = __half_as_ushort(__float2half_rn(d));
    const uint32_t s16 = __half_as_ushort(__float2half_rn(__fmul_rn(d, static_cast<float>(sum))));
    blk[0] = d16 | (s16 << 16);
  }
}

__device__ __forceinline__ float mean_of(float sum, int k, float eps) { return __fadd_rn(__fdiv_rn(sum, static_cast<float>(k)), eps); }
// 1 / sqrt(mean); a row of zeros stays one.
__device__ __forceinline__ float inverse_root(float mean) {
  return mean > 0.0f ? __frcp_rn(__fsqrt_rn(mean)) : (mean == 0.0f ? 0.0f : mean);
}

// What a row is multiplied by, and its sum formed anew, where the squares of
// its values leave fp32's range.  Up: below 2^-100 of a mean, what squares
// below 2^-126 lose (2^-150 each) would no longer be lost beside it; values, at most
// 2^-50 sqrt(k), then lie in 2^-49 .. 2^60.  Down: values lie below 2^53, their
// squares' sum below 2^126; those that lose bits are below 2^-126 in y.
__device__ __forceinline__ float factor_of(float mean) {
  if (mean < 7.888609052210118e-31f) return 1.2676506002282294e30f;   // 2^-100: 2^100
  return mean == INFINITY ? 2.6469779601696886e-23f : 1.0f;            // 2^-75; NaN stays
}
__device__ __forceinline__ Eight times(const Eight& v, float by) {
  return {make_float4(v.a.x * by, v.a.y * by, v.a.z * by, v.a.w * by), make_float4(v.b.x * by, v.b.y * by, v.b.z * by, v.b.w * by)};
}

// The sum over a block, by all threads, through `part`, which the threads may
// read until the block's next barrier.
__device__ __forceinline__ float block_sum(float sum, float* part) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = lane < (blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// A row once more, by all threads, if its squares leave fp32's range: read from
// where it is (x' where that has been stored).  Not inlined, and for rows copied
// ahead behind the others: such a branch among them costs all rows (4096 of 5120
// with a bf16 delta 43.5 us, with the branch in the loop 44.5).
template <typename TD>
__device__ __noinline__ void far_row(const RowOf r, int k, float eps, float* part) {
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x, groups = k >> 3;
  auto load = [&](int i) { return r.x_out ? load8(r.x_out, i) : load_x<TD>(r, i); };
  float by = 1.0f, mean;
  for (;;) {
    float sum = 0.0f;
#pragma unroll 1
    for (int i = tid; i < groups; i += threads) sum = square_sum(times(load(i), by), sum);
    __syncthreads();  // part may still be read
    mean = mean_of(block_sum(sum, part), k, eps * by * by);
    if (by != 1.0f) break;
    by = factor_of(mean);
    if (by == 1.0f) return;
  }
  const float inv = inverse_root(mean);
#pragma unroll 1
  for (int i = tid; i - lane < groups; i += threads) {
    Eight w = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (i < groups) w = times(load(i), by);
    finish(r, i, i < groups, w, inv);
  }
}

template <typename TD, int NV>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a, int one_wave) {
  __shared__ float s_part[32];
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const int groups = a.k >> 3;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * a.k;
  RowOf r;
  r.x = a.x + at;
  if constexpr (!std::is_same<TD, NoDelta>::value) r.delta = static_cast<const TD*>(a.delta) + at;
  r.gamma = a.gamma;
  r.x_out = a.x_out ? a.x_out + at : nullptr;
  r.q8 = a.q8 ? a.q8 + static_cast<int64_t>(blockIdx.x) * (a.k >> 5) * 9 : nullptr;
  r.y = a.y ? static_cast<uint8_t*>(a.y) + at * (a.y_type == kF32 ? 4 : 2) : nullptr;
  r.y_type = a.y_type;
  if (one_wave) pdl_launch_dependents();
  pdl_wait();
  Eight v[NV > 0 ? NV : 1];
  float sum = 0.0f;
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * threads;
      v[j] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      if (i < groups) v[j] = load_x<TD>(r, i);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (r.x_out && tid + j * threads < groups) store_x(r, tid + j * threads, v[j]);
      sum = square_sum(v[j], sum);
    }
  } else {
    for (int i = tid; i < groups; i += threads) {
      const Eight w = load_x<TD>(r, i);
      if (r.x_out) store_x(r, i, w);
      sum = square_sum(w, sum);
    }
  }
  sum = block_sum(sum, s_part);
  float mean = mean_of(sum, a.k, a.eps);
  const float by = factor_of(mean);
  if (by != 1.0f) {  // of all threads
    sum = 0.0f;
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[j] = times(v[j], by);
        sum = square_sum(v[j], sum);
      }
    } else {
      far_row<TD>(r, a.k, a.eps, s_part);
      return;
    }
    __syncthreads();
    mean = mean_of(block_sum(sum, s_part), a.k, a.eps * by * by);
  }
  const float inv = inverse_root(mean);
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * threads;
      finish(r, i, i < groups, v[j], inv);
    }
  } else {
    for (int i = tid; i - lane < groups; i += threads) {
      Eight w = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      // What this thread stored above where it did: x may be x_out.
      if (i < groups) w = r.x_out ? load8(r.x_out, i) : load_x<TD>(r, i);
      finish(r, i, i < groups, w, inv);
    }
  }
}

// Many long rows: persistent CTAs whose next rows are copied to shared memory while
// one is worked on.  A row's slot is free as soon as its values are in
// registers, which the barrier of the sum says, so a row takes one barrier.
template <typename TD, int NV>
__global__ void __launch_bounds__(NV == 2 ? 512 : 544, NV == 2 ? 2 : 1) rms_norm_rows_kernel(const NormArgs a, int64_t t, unsigned* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kSlots];
  __shared__ float s_part[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int groups = a.k >> 3;
  const uint32_t x_bytes = static_cast<uint32_t>(a.k) * 4, d_bytes = static_cast<uint32_t>(a.k) * delta_size<TD>();
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  auto fetch = [&](int64_t row, int slot) {  // thread 0
    asm volatile("fence.proxy.async;" ::: "memory");  // behind the call before, and the reads of the row that was here
    uint8_t* to = smem + slot * (x_bytes + d_bytes);
    mbar_arrive_expect_tx(&bars[slot], x_bytes + d_bytes);
    bulk_g2s_nohint(to, a.x + row * a.k, x_bytes, &bars[slot]);
    bulk_g2s_nohint(to + x_bytes, static_cast<const TD*>(a.delta) + row * a.k, d_bytes, &bars[slot]);
  };
  if (tid == 0)
    for (int i = 0; i < kSlots; ++i)
      if (blockIdx.x + static_cast<int64_t>(i) * gridDim.x < t) fetch(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
  int slot = 0;
  uint32_t phase = 0;
  bool far = false;  // whether a row is left for the end; the same for all threads
#pragma unroll 1
  for (int64_t row = blockIdx.x, turn = 0; row < t; row += gridDim.x, ++turn) {
    RowOf r = row_of<TD>(a, row);
    r.x = reinterpret_cast<const float*>(smem + slot * (x_bytes + d_bytes));
    r.delta = smem + slot * (x_bytes + d_bytes) + x_bytes;
    const bool ok = mbar_wait(&bars[slot], phase);
    Eight v[NV];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * threads;
      v[j] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      if (i < groups) v[j] = load_x<TD>(r, i);
      sum = square_sum(v[j], sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_part[turn & 1][warp] = sum;
    if (__syncthreads_or(!ok)) {
      if (tid == 0) {
        raise_status(status, kStatusTimeout);
        for (int i = 0; i < kSlots; ++i) (void)mbar_wait(&bars[i], phase);  // let copies land (bounded)
      }
      return;
    }
    if (tid == 0 && row + kSlots * static_cast<int64_t>(gridDim.x) < t) fetch(row + kSlots * static_cast<int64_t>(gridDim.x), slot);
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
    sum = lane < (threads >> 5) ? s_part[turn & 1][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float mean = mean_of(sum, a.k, a.eps);
    far |= factor_of(mean) != 1.0f;
    const float inv = inverse_root(mean);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * threads;
      if (r.x_out && i < groups) store_x(r, i, v[j]);
      finish(r, i, i < groups, v[j], inv);
    }
  }
  if (far)
    for (int64_t row = blockIdx.x; row < t; row += gridDim.x) far_row<TD>(row_of<TD>(a, row), a.k, a.eps, s_part[0]);
}

template <typename TD, int NV>
int launch_rows(const NormArgs& a, int64_t t, int threads, unsigned* status, cudaStream_t s) {
  const int64_t smem = kSlots * static_cast<int64_t>(a.k) * (4 + delta_size<TD>());
  static std::atomic<bool> configured[64];  // per device (racing threads configure twice: idempotent)
  const DeviceInfo& di = device_info();
  if (di.device < 0 || di.device >= 64) return TQ1_ERR_CUDA;
  if (!configured[di.device].load(std::memory_order_acquire)) {
    if (!cuda_ok(cudaFuncSetAttribute(rms_norm_rows_kernel<TD, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRowsSmem))))
      return TQ1_ERR_CUDA;
    configured[di.device].store(true, std::memory_order_release);
  }
  const int64_t fit = std::min<int64_t>(std::min<int64_t>(1024 / threads, 228 * 1024 / (smem + 1024)), 6);
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(t, std::max<int64_t>(1, fit) * std::max(1, di.num_sms))));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, rms_norm_rows_kernel<TD, NV>, a, t, status)) ? TQ1_OK : TQ1_ERR_CUDA;
}

template <typename TD, int NV>
int launch(const NormArgs& a, int64_t t, int threads, int one_wave, cudaStream_t s) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(t));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, rms_norm_kernel<TD, NV>, a, one_wave)) ? TQ1_OK : TQ1_ERR_CUDA;
}

template <typename TD>
int launch_delta(const NormArgs& a, int64_t t, unsigned* status, cudaStream_t s) {
  const int sms = std::max(1, device_info().num_sms);
  const int groups = a.k >> 3;
  auto threads_of = [&](int nv) { return ((groups + nv - 1) / nv + 31) / 32 * 32; };
  auto resident = [&](int nv) { return static_cast<int64_t>(sms) * ((nv == 1 ? 2048 : nv == 2 ? 1344 : 1024) / threads_of(nv)); };
  // Rows copied ahead, where a row with its delta is 36 KB and more and there are
  // several to a CTA, unless only one such CTA fits an SM where the other kernel has
  // two rows.  With a 16-bit delta, not so and so: 4096 rows of 2048 18.2 and 20.1 us,
  // of 4096 34.0 and 34.6; 2432 of 6144 32.7 and 32.5; 6000 of 8192 100 and 91; 4096 of
  // 10240 82 and 99, of 11264 121 and 110.  With an fp32 delta slower (4096 rows of
  // 6144 52 and 60, of 12288 119 and 132), and without one (of 5120 26.4 and 28.5): not there.
  if constexpr (delta_size<TD>() == 2) {
    const int64_t smem = kSlots * static_cast<int64_t>(a.k) * 6;
    if (t >= 8 * sms && a.k >= kRowsMinK && smem <= kRowsSmem && (2 * (smem + 1024) <= 228 * 1024 || resident(2) < 2 * sms)) {
      if (groups <= 2 * 512) return launch_rows<TD, 2>(a, t, ((groups + 1) / 2 + 31) / 32 * 32, status, s);
      return launch_rows<TD, 4>(a, t, ((groups + 3) / 4 + 31) / 32 * 32, status, s);
    }
  }
  // Groups of a thread: the fewest with which all rows are resident at once (a
  // thread has 32, 48 or 64 registers), but two where one makes CTAs of 800 threads and more.
  // One, two and four groups, with an fp32 delta: 48 rows of 2080 2.3, 2.8 and 3.7 us, 517 of them
  // 4.6, 5.0 and 6.1, 1000 rows of 1024 4.2, 4.6 and 5.8; 48 rows of 8192 4.9, 4.8 and 5.8, 400 of
  // them 10.6, 10.7 and 10.6.  Beyond that two (3000 rows of 5120 33.5, 33.9 and 38.2, 4096 of them
  // without a delta 31.6, 26.8 and 26.6), unless four take two waves where two take more than
  // three (1000 rows of 8192 21.4, 20.9 and 23.2, without a delta 16.0, 14.9 and 13.5).
  int nv = 2;
  if (groups <= 768 && t <= resident(1)) nv = 1;
  else if (t > resident(2) && (t <= resident(4) || (t > 3 * resident(2) && t <= 2 * resident(4)))) nv = 4;
  while (nv < 4 && threads_of(nv) > 1024) nv *= 2;
  if (threads_of(nv) > 1024) nv = 0;
  const int threads = nv ? threads_of(nv) : 1024;
  const int one_wave = t <= sms;
  switch (nv) {
    case 1: return launch<TD, 1>(a, t, threads, one_wave, s);
    case 2: return launch<TD, 2>(a, t, threads, one_wave, s);
    case 4: return launch<TD, 4>(a, t, threads, one_wave, s);
    default: return launch<TD, 0>(a, t, threads, one_wave, s);
  }
}

}  // namespace

int launch_rms_norm(const NormArgs& a, int64_t t, unsigned* status, cudaStream_t s) {
  if (!a.delta) return launch_delta<NoDelta>(a, t, status, s);
  switch (a.delta_type) {
    case kF16: return launch_delta<__half>(a, t, status, s);
    case kBf16: return launch_delta<__nv_bfloat16>(a, t, status, s);
    default: return launch_delta<float>(a, t, status, s);
  }
}

}  // namespace tq1
