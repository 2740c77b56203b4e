// The norm in front of the head and the 8-bit (e4m3) formats of the 8-bit
// dense head:
//  * rmsnorm: t = x + r, y = t / sqrt(mean(t^2) + eps) * (offset + w) per
//    row, t and y rounded once to the storage type, and/or y in e4m3 with one
//    fp32 scale per 128 columns;
//  * quantize_fp8: a matrix in e4m3 with one fp32 scale per 128 x 128 block.
// Scale of a block: max(max|y| / 448, 2^-126); code: e4m3 of y / scale, to
// nearest, ties to even.  The floor keeps the scale a normal number, so that
// y / scale stays exact enough for tiny blocks and a zero block divides by no
// zero.
#include "fh_device.h"
#include "fh_internal.h"

namespace fh {

namespace {

constexpr int kNormThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126

// One 16-byte chunk of a row: 8 bf16 or 4 fp32 values.
template <typename T> struct Unit;
template <> struct Unit<bf16_t> {
  static constexpr int kElems = 8;
  __device__ __forceinline__ static void load(const uint8_t* p, float* v) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
  }
  __device__ __forceinline__ static uint32_t pair(float a, float b) {
    return (uint32_t)f32_to_bf16_rne(a) | ((uint32_t)f32_to_bf16_rne(b) << 16);
  }
  __device__ __forceinline__ static void store(uint8_t* p, const float* v) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
  }
};
template <> struct Unit<float> {
  static constexpr int kElems = 4;
  __device__ __forceinline__ static void load(const uint8_t* p, float* v) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
  __device__ __forceinline__ static void store(uint8_t* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// four codes in one word (values within the format's range after the scale)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ float block_scale(float amax) {
  return fmaxf(amax / kE4m3Max, kScaleFloor);
}

// largest value over the lanes of each aligned group of `lanes` (a power of two)
template <int lanes>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) x = fmaxf(x, __shfl_xor(x, o, kWave));
  return x;
}

template <int n>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* q) {
  if constexpr (n == 8)
    *reinterpret_cast<uint2*>(p) =
        make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
  else
    *reinterpret_cast<uint32_t*>(p) = e4m3x4(q[0], q[1], q[2], q[3]);
}

// From this mean of squares on, with eps, the roundings of squares and sums below
// 2^-126 (by up to 2^-150 each) are nothing beside a row's sum.
constexpr float kSmallMean = 7.88860905e-31f;  // 2^-100

// kRowThreads threads per row (a wave, four rows a workgroup, or the whole
// workgroup); the row stays in registers between the sum and the outputs, so x
// may be y and r may be the residual's output.  Bound by memory: 8192 rows of
// 2048 bf16 with the residual, to 8 bits, take 25.6 to 28.3 us for 118 MB (4.2 to
// 4.6 TB/s; a large copy reaches 5.1), of fp32 44 us for 219 MB (5.0).
template <typename T, int kRowThreads, int kUnits>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_kernel(const RmsnormArgs a) {
  constexpr int N = Unit<T>::kElems;
  constexpr int kGroupLanes = 128 / N;  // lanes that hold one block of 128 columns
  constexpr int kRows = kNormThreads / kRowThreads;
  __shared__ float s_sum[kNormThreads / kWave];
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kRowThreads;
  const int tid = threadIdx.x % kRowThreads;
  if (kRows > 1 && row >= a.rows) return;  // (a whole wave)
  const uint8_t* x = a.x + row * a.x_bytes;
  float t[kUnits][N];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = i * kRowThreads + tid;
    if (u < a.units) {
      Unit<T>::load(x + (int64_t)u * 16, t[i]);
      if (a.r) {
        float r[N];
        Unit<T>::load(a.r + row * a.r_bytes + (int64_t)u * 16, r);
#pragma unroll
        for (int j = 0; j < N; ++j) t[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) t[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) ss = fmaf(t[i][j], t[i][j], ss);
  }
  float tot = wave_sum(ss);
  if constexpr (kRows == 1) {
    if ((tid & (kWave - 1)) == 0) s_sum[tid / kWave] = tot;
    __syncthreads();
    tot = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / kWave; ++w) tot += s_sum[w];
  }
  const float mean = tot / (float)a.d + a.eps;
  float rstd = 1.0f / sqrtf(mean);
  const bool wide = !(mean >= kSmallMean && mean < INFINITY);
  if (wide) {
    // The squares leave the range of fp32: the same in fp64, where they do not.
    // Also 1 / sqrt(mean) may be out of range where t times it is not.
    __shared__ double s_wide[kNormThreads / kWave];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        sum = fma((double)t[i][j], (double)t[i][j], sum);
        asm volatile("" : "+v"(t[i][j]));  // (not kept in fp64 for the loop below)
      }
    }
    for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    if constexpr (kRows == 1) {  // (the mean, and so this branch, is the workgroup's)
      if ((tid & (kWave - 1)) == 0) s_wide[tid / kWave] = sum;
      __syncthreads();
      sum = 0.0;
      for (int w = 0; w < kNormThreads / kWave; ++w) sum += s_wide[w];
    }
    const double r = 1.0 / sqrt(sum / (double)a.d + (double)a.eps);
    rstd = 1.0f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = i * kRowThreads + tid;
      if (a.r_out && u < a.units)
        Unit<T>::store(a.r_out + row * a.ro_bytes + (int64_t)u * 16, t[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) t[i][j] = (float)((double)t[i][j] * r);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = i * kRowThreads + tid;
    const bool in = u < a.units;
    float y[N];
    if (in) {
      if (a.r_out && !wide) Unit<T>::store(a.r_out + row * a.ro_bytes + (int64_t)u * 16, t[i]);
      float w[N];
      if (a.w) Unit<T>::load(a.w + (int64_t)u * 16, w);
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = t[i][j] * rstd * ((a.w ? w[j] : 1.0f) + a.offset);
      if (a.y) Unit<T>::store(a.y + row * a.y_bytes + (int64_t)u * 16, y);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = 0.0f;
    }
    if (a.y8) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(y[j]));
      const float s = block_scale(group_max<kGroupLanes>(m));
      if (in) {
        float q[N];
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = y[j] / s;
        store_codes<N>(a.y8 + row * a.ldy8 + (int64_t)u * N, q);
        if (u % kGroupLanes == 0) a.scale[row * a.lds + u / kGroupLanes] = s;
      }
    }
  }
}

// One workgroup per 128 x 128 block, held in registers between the maximum
// and the codes.  Bound by memory: 128256 x 2048 bf16 take 149 us for 788 MB
// (5.3 TB/s), with IEEE divisions.
template <typename T>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(const QuantizeFp8Args a) {
  constexpr int N = Unit<T>::kElems;
  constexpr int kLanes = 128 / N;         // lanes along a row of the block
  constexpr int kRows = 256 / kLanes;     // rows per step
  constexpr int kSteps = 128 / kRows;
  __shared__ float s_max[256 / kWave];
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * 128 + tid / kLanes;
  const int col = blockIdx.x * 128 + (tid % kLanes) * N;
  const bool cin = col < a.d;
  float t[kSteps][N];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * kRows;
    if (cin && r < a.v) {
      Unit<T>::load(a.E + r * a.e_bytes + (int64_t)col * (16 / N), t[i]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) t[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(t[i][j]));
  }
  m = wave_max(m);
  if ((tid & (kWave - 1)) == 0) s_max[tid / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 256 / kWave; ++w) m = fmaxf(m, s_max[w]);
  const float s = block_scale(m);
  if (tid == 0) a.scale[(int64_t)blockIdx.y * a.lds + blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * kRows;
    if (cin && r < a.v) {
      float q[N];
#pragma unroll
      for (int j = 0; j < N; ++j) q[j] = t[i][j] / s;
      store_codes<N>(a.codes + r * a.ldc + col, q);
    }
  }
}

template <typename T>
void enqueue_rmsnorm(const RmsnormArgs& a, hipStream_t s) {
  const dim3 block(kNormThreads);
  const dim3 each((unsigned)a.rows), four((unsigned)((a.rows + 3) / 4));
  // A wave per row where one chunk a lane holds it (8192 x 256 bf16: 6.6 us, 9.4
  // with a workgroup per row); with two a lane it is slower (8192 x 1024: 15.2,
  // 13.9).
  if (a.units <= kWave)
    hipLaunchKernelGGL((rmsnorm_kernel<T, kWave, 1>), four, block, 0, s, a);
  else if (a.units <= kNormThreads)
    hipLaunchKernelGGL((rmsnorm_kernel<T, kNormThreads, 1>), each, block, 0, s, a);
  else if (a.units <= 2 * kNormThreads)
    hipLaunchKernelGGL((rmsnorm_kernel<T, kNormThreads, 2>), each, block, 0, s, a);
  else if (a.units <= 4 * kNormThreads)
    hipLaunchKernelGGL((rmsnorm_kernel<T, kNormThreads, 4>), each, block, 0, s, a);
  else if constexpr (sizeof(T) == 4)
    hipLaunchKernelGGL((rmsnorm_kernel<T, kNormThreads, 8>), each, block, 0, s, a);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormArgs& a, int dtype, hipStream_t s) {
  if (dtype == FH_DTYPE_BF16)
    enqueue_rmsnorm<bf16_t>(a, s);
  else
    enqueue_rmsnorm<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_quantize_fp8(const QuantizeFp8Args& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)((a.d + 127) / 128), (unsigned)((a.v + 127) / 128));
  if (dtype == FH_DTYPE_BF16)
    hipLaunchKernelGGL(quantize_fp8_kernel<bf16_t>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(quantize_fp8_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace fh
