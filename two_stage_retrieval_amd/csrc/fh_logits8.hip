// Logits of the 8-bit dense head:
//   z[m, t] = sum_g hs[m, g] es[t / 128, g] sum_{k in block g} h8[m, k] e8[t, k]
// over e4m3 codes, one fp32 scale per 128 columns of a row of h and per
// 128 x 128 block of E.  The products of a block of 128 columns are summed by
// the matrix cores; its fp32 result is then scaled and added to the fp32
// accumulator, since the scales change from block to block.
#include "fh_device.h"
#include "fh_internal.h"

namespace fh {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 8 codes as bf16 values (exact: e4m3 has fewer bits in both fields)
__device__ __forceinline__ v8bf to_bf16(int w0, int w1) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// D[i, j] = sum over 128 columns of A[i, :] . B[j, :], 16 x 16.  Lane l gives
// 32 bytes of row l % 16 of A and of B (any order of the columns that both
// share); it receives rows 4 (l / 16) + 0..3 of column l % 16.
//
// The codes go through the bf16 instruction: the 8-bit one drops, within
// small groups of products, the bits far below the group's largest product
// (on codes spread over the format's range its sums were 4.5e-5 off, against
// 3e-8 for the bf16 instruction).
__device__ __forceinline__ v4f mfma128(v8i a, v8i b) {
  v4f c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(a[i], a[i + 1]), to_bf16(b[i], b[i + 1]),
                                                c, 0, 0, 0);
  return c;
}

// the 32 bytes of a row's block that lane quarter q gives: [16 q, 16 q + 16)
// and the same 64 bytes on, zero past the row's end
__device__ __forceinline__ v8i load_block(const uint8_t* row, int k, int d) {
  v4i lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (k < d) lo = *reinterpret_cast<const v4i*>(row + k);
  if (k + 64 < d) hi = *reinterpret_cast<const v4i*>(row + k + 64);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One wave per 16 rows of E and 16 rows of h.
template <typename TO>
__global__ __launch_bounds__(256) void logits8_kernel(const Logits8Args a) {
  const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 16;
  const int m0 = blockIdx.y * 16;
  if (n0 >= a.v) return;
  const int64_t n = n0 + c < a.v ? n0 + c : a.v - 1;
  const int m = m0 + c < a.rows ? m0 + c : a.rows - 1;
  const uint8_t* e = a.E8 + n * a.lde;
  const uint8_t* h = a.h8 + (int64_t)m * a.ldh;
  const float* hs = a.h_scale + (int64_t)m * a.lds;
  const float* es = a.E_scale + (n0 / 128) * a.ldes;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < a.d; k += 128) {
    const v4f p = mfma128(load_block(e, k + 16 * q, a.d), load_block(h, k + 16 * q, a.d));
    const float s = hs[k / 128] * es[k / 128];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
  }
  if (m0 + c >= a.rows) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = n0 + 4 * q + i;
    if (t < a.v) {
      if constexpr (sizeof(TO) == 4)
        reinterpret_cast<float*>(a.out)[(int64_t)m * a.ldo + t] = acc[i];
      else
        reinterpret_cast<uint16_t*>(a.out)[(int64_t)m * a.ldo + t] = f32_to_bf16_rne(acc[i]);
    }
  }
}

}  // namespace

hipError_t launch_logits8(const Logits8Args& a, int out_dtype, hipStream_t s) {
  const dim3 grid((unsigned)((a.v + 63) / 64), (unsigned)((a.rows + 15) / 16));
  if (out_dtype == FH_DTYPE_BF16)
    hipLaunchKernelGGL(logits8_kernel<uint16_t>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(logits8_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace fh
