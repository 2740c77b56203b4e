// Loads of rows of either storage type, and pieces of sums over a row of logits in
// fp64: the weight of a value, and sums over a wave.
#pragma once
#include "fh_device.h"

namespace fh {

// Running sum over the wave, in lane order, on DPP (both words of a value move
// by the same control; lanes without a source add 0).  Every lane is active.
__device__ __forceinline__ double wave_scan_f64(double x) {
#define FH_DPP_ADD(ctrl, rmask)                                                                 \
  x += __hiloint2double(                                                                        \
      __builtin_amdgcn_update_dpp(0, __double2hiint(x), ctrl, rmask, 0xf, false),               \
      __builtin_amdgcn_update_dpp(0, __double2loint(x), ctrl, rmask, 0xf, false));
  FH_DPP_ADD(0x111, 0xf)  // row_shr:1
  FH_DPP_ADD(0x112, 0xf)  // row_shr:2
  FH_DPP_ADD(0x114, 0xf)  // row_shr:4
  FH_DPP_ADD(0x118, 0xf)  // row_shr:8
  FH_DPP_ADD(0x142, 0xa)  // row_bcast:15 into rows 1 and 3
  FH_DPP_ADD(0x143, 0xc)  // row_bcast:31 into rows 2 and 3
#undef FH_DPP_ADD
  return x;
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), lane),
                          __builtin_amdgcn_readlane(__double2loint(x), lane));
}
__device__ __forceinline__ double wave_sum_f64(double x) { return lane_f64(wave_scan_f64(x), 63); }

// 2^((x - top) k) for x <= top, not NaN; kZero: 0 from 2^-1020 on, else at
// least about that (enough for a sum that holds a 1; lo = -1020 / k).  With
// (x - top) k = n + f, n the nearest whole number, it is 2^f with n added to the
// exponent; n is the low word of a sum with 1.5 * 2^52, and 2^f is 1 + f r(f), r
// the polynomial that interpolates (2^f - 1) / f at the nine Chebyshev nodes of
// [-1/2, 1/2] (relative error below 4e-14).  The weight of the largest value is
// 1 itself, so that the running sums over equal largest values are whole numbers
// and a uniform number on a border between two of them falls on the right side.
// These instructions set the time of the first launch: 17 a value, about 1 us
// each for 288 rows of 128256, which take 31 us in all where reading them takes
// 14 (80 with the library's exp, 42 with conversions to and from n; requesting
// the next values before these are summed changes nothing).
template <bool kZero = true>
__device__ __forceinline__ double weight(float x, float top, double k, double lo = 0.0) {
  double d = (double)x - (double)top;
  if constexpr (!kZero) d = fmax(d, lo);
  const double n = fma(d, k, 6755399441055744.0), f = fma(d, k, 6755399441055744.0 - n);
  double p = 1.02031210633917290e-07;
  p = fma(p, f, 1.32552248786688168e-06);
  p = fma(p, f, 1.52526868462677196e-05);
  p = fma(p, f, 1.54034558524538382e-04);
  p = fma(p, f, 1.33335581790431116e-03);
  p = fma(p, f, 9.61812915940255843e-03);
  p = fma(p, f, 5.55041086647604237e-02);
  p = fma(p, f, 2.40226506958129887e-01);
  p = fma(p, f, 6.93147180559945286e-01);
  p = fma(p, f, 1.0);
  p = __hiloint2double(__double2hiint(p) + (__double2loint(n) << 20), __double2loint(p));
  if constexpr (kZero) p = n < 6755399441055744.0 - 1020.0 ? 0.0 : p;
  return p;
}

// The largest of three numbers from memory in one instruction (fmaxf takes another
// for each of them).  A quiet NaN is left out; a signalling one comes out quiet, and
// with it what was largest until then is lost: callers look for NaNs themselves.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Values [i, i + 8) of a row.
template <typename T>
__device__ __forceinline__ void load_whole8(const uint8_t* row, int64_t i, float* x) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + i * 2);
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(row + i * 4);
    const float4 b = *reinterpret_cast<const float4*>(row + i * 4 + 16);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}
// The same of a row of n: past its end `fill`, without reading there.
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* row, int64_t i, int64_t n, float fill,
                                      float* x) {
  if (i + 8 <= n) {
    load_whole8<T>(row, i, x);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = fill;
    if (i + j < n) {
      if constexpr (sizeof(T) == 2)
        x[j] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i + j] << 16);
      else
        x[j] = reinterpret_cast<const float*>(row)[i + j];
    }
  }
}

template <typename T>
__device__ __forceinline__ float load1(const uint8_t* row, int64_t i) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  else
    return reinterpret_cast<const float*>(row)[i];
}

}  // namespace fh
