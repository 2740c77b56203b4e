// The dense head in 4 bits: E's codes with a bf16 scale (and zero) per group of
// 32, 64 or 128 columns of a row, rows read back from them, and the logits
//   z[m, t] = sum_g s[g, t] sum_{k in g} (q[t, k] - zero[g, t]) h[m, k].
#include "fh_device.h"
#include "fh_host.h"
#include "fh_internal.h"
#include "fh_weights.h"

namespace fh {

namespace {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// E to 4 bits
// ---------------------------------------------------------------------------

// The largest |.|, and the smallest, of three, as max3 does.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// x / s rounded, for a bf16 number s, in three instructions for each x instead of
// the ten of a division: the reciprocal is refined to the nearest one (from any
// within one step, for each of the 128 fractions of s), and the quotient by its
// remainder.  What is made of it is the nearest whole number, so only quotients
// near k + 1/2 matter; for all of those within four steps it is the rounded one
// (checked one by one).  Nothing leaves the normal numbers for s in [2^-90, 2^100]
// and x up to 15 s.
__device__ __forceinline__ float reciprocal(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return fmaf(fmaf(-s, r, 1.0f), r, r);
}
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q);
}

// the word of 8 columns' codes
__device__ __forceinline__ uint32_t pack8(const int* q) {
  uint32_t b[4];   // bytes: columns 0 and 2, 4 and 6, 1 and 3, 5 and 7
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = (i & 1) * 4 + (i >> 1);
    b[i] = ((uint32_t)q[j] & 15u) | ((uint32_t)q[j + 2] << 4);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400);
  const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400);
  return lo | hi << 16;
}

// a whole number cut to [-8, 7]; 0 for a NaN
__device__ __forceinline__ float cut4(float x) {
  return x == x ? fminf(fmaxf(x, -8.0f), 7.0f) : 0.0f;
}

// The largest x, or the sum, of the 4, 8 or 16 neighbouring lanes of a group, on
// DPP: swaps within four lanes, then mirrored halves, whose lanes hold the same
// value by then.
template <int kLanes, typename Op>
__device__ __forceinline__ float group_reduce(float x, Op op) {
#define FH_DPP_GROUP(ctrl) \
  x = op(x, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), ctrl, 0xf, 0xf, true)))
  FH_DPP_GROUP(0xB1);                               // quad_perm 1 0 3 2
  FH_DPP_GROUP(0x4E);                               // quad_perm 2 3 0 1
  if constexpr (kLanes >= 8) FH_DPP_GROUP(0x141);   // row_half_mirror
  if constexpr (kLanes >= 16) FH_DPP_GROUP(0x140);  // row_mirror
#undef FH_DPP_GROUP
  return x;
}
template <int kLanes>
__device__ __forceinline__ float group_max(float x) {
  return group_reduce<kLanes>(x, [](float a, float b) { return fmaxf(a, b); });
}
template <int kLanes>
__device__ __forceinline__ float group_sum(float x) {
  return group_reduce<kLanes>(x, [](float a, float b) { return a + b; });
}

// One workgroup per 64 rows by 128 columns, held in registers between the
// maxima and the codes: 16 lanes a row.  The scales of 64 rows are joined in
// LDS, since a group's scales lie along the rows.  128256 x 2048 bf16 take 169 us for
// 660 MB (3.9 TB/s): the vector instructions alone are 115 of them, the memory 127 at
// a copy's rate (with IEEE divisions 230 us).
template <typename T, int kGroup, bool kZero>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const QuantizeInt4Args a) {
  constexpr int kRows = 64, kSteps = kRows / 16, kSubs = 128 / kGroup, kLanes = kGroup / 8;
  __shared__ uint16_t s_scale[kSubs][kRows], s_zero[kSubs][kRows];
  const int tid = threadIdx.x, in = tid >> 4, u = tid & 15;
  // (neighbouring workgroups: neighbouring columns)
  const unsigned across = (unsigned)(a.d + 127) / 128, block = blockIdx.x % across;
  const int64_t r0 = (int64_t)(blockIdx.x / across) * kRows;
  const int col = block * 128 + u * 8;
  const bool cin = col < a.d;
  float x[kSteps][8];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * 16 + in;
    if (cin && r < a.v) {
      load_whole8<T>(a.E + r * a.e_bytes, col, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * 16 + in;
    float hi = 0.0f, lo = 0.0f, zero = 0.0f, scale;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      nan |= __builtin_isunordered(x[i][j], x[i][j + 1]);
      hi = kZero ? max3(hi, x[i][j], x[i][j + 1]) : max3_abs(hi, x[i][j], x[i][j + 1]);
      if constexpr (kZero) lo = min3(lo, x[i][j], x[i][j + 1]);
    }
    if (nan) {
      hi = lo = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[i][j] == x[i][j] ? x[i][j] : 0.0f;
        hi = fmaxf(hi, kZero ? y : fabsf(y));
        if constexpr (kZero) lo = fminf(lo, y);
      }
    }
    hi = group_max<kLanes>(hi);
    if constexpr (kZero) {
      lo = group_max<kLanes>(-lo);
      scale = hi / 15.0f + lo / 15.0f;
    } else {
      scale = hi / 7.0f;
    }
    const uint16_t bits = f32_to_bf16_rne(fmaxf(scale, 0x1p-126f));
    scale = __uint_as_float((uint32_t)bits << 16);
    if constexpr (kZero) zero = cut4(-8.0f + rintf(lo / scale));
    if (u % kLanes == 0) {
      s_scale[u / kLanes][i * 16 + in] = bits;
      if constexpr (kZero)   // (a whole number of 4 bits is a bf16 value)
        s_zero[u / kLanes][i * 16 + in] = (uint16_t)(__float_as_uint(zero) >> 16);
    }
    int q[8];   // (the lower 4 bits count)
    if (!nan && scale >= 0x1p-90f && scale <= 0x1p100f) {
      const float inv = reciprocal(scale);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = quotient(x[i][j], scale, inv);
        q[j] = (int)__float_as_uint(__builtin_amdgcn_fmed3f(y, -8.0f - zero, 7.0f - zero) +
                                    12582912.0f);   // 1.5 * 2^23: the nearest whole number
        if constexpr (kZero) q[j] += (int)zero;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = (int)cut4(rintf(x[i][j] / scale) + zero);
    }
    if (cin && r < a.v)
      *reinterpret_cast<uint32_t*>(a.codes + r * a.c_bytes + col / 2) = pack8(q);
  }
  __syncthreads();
  const int sub = tid >> 6, row = tid & 63;
  const int g = block * kSubs + sub;
  if (sub < kSubs && g * kGroup < a.d && r0 + row < a.v) {
    a.scale[g * a.lds + r0 + row] = s_scale[sub][row];
    if constexpr (kZero) a.zero[g * a.lds + r0 + row] = s_zero[sub][row];
  }
}

template <typename T, int kGroup>
void enqueue_quantize(const QuantizeInt4Args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.v + 63) / 64 * ((a.d + 127) / 128)));
  if (a.zero)
    hipLaunchKernelGGL((quantize_int4_kernel<T, kGroup, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((quantize_int4_kernel<T, kGroup, false>), grid, dim3(256), 0, s, a);
}

// ---------------------------------------------------------------------------
// rows read back
// ---------------------------------------------------------------------------

// the code of column 8 i + j in the word of columns 8 i .. 8 i + 7
__device__ __forceinline__ float code_at(uint32_t w, int j) {
  return (float)((int32_t)(w << (28 - 4 * (j / 2 + 4 * (j & 1)))) >> 28);
}

// A wave takes 8 rows, 8 columns a lane; all that it reads is requested before
// the first row is written (rows of two dependent reads each would follow one another
// otherwise).  Bound by memory for rows in a row (128256 x 2048 to bf16: 112 us, 5.9
// TB/s) and, by ids, by the lines that the scales lie in: a token's 2 bytes bring
// 63 other tokens' with them, once a group.
constexpr int kReadRows = 8;
template <typename TO, bool kZero>
__global__ __launch_bounds__(256) void int4_rows_kernel(const Int4RowsArgs a, int shift) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const unsigned across = (unsigned)(a.E.d + 511) / 512;
  const int col = blockIdx.x % across * 512 + lane * 8;
  if (col >= a.E.d) return;
  const uint16_t* scale = a.E.scale + (int64_t)(col >> shift) * a.E.lds;
  const uint16_t* zero = kZero ? a.E.zero + (int64_t)(col >> shift) * a.E.lds : nullptr;
  const int64_t r0 = ((int64_t)(blockIdx.x / across) * 4 + w) * kReadRows;
  if (r0 >= a.rows) return;
  int64_t id[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int64_t r = r0 + i < a.rows ? r0 + i : a.rows - 1;
    id[i] = a.ids ? (int64_t)a.ids[r] : r;
  }
  uint32_t q[kReadRows];
  uint16_t s[kReadRows], z[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int64_t t = id[i] >= 0 && id[i] < a.E.v ? id[i] : 0;
    q[i] = *reinterpret_cast<const uint32_t*>(a.E.codes + t * a.E.c_bytes + col / 2);
    s[i] = scale[t];
    z[i] = kZero ? zero[t] : (uint16_t)0;
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (r0 + i >= a.rows) return;
    const bool in = id[i] >= 0 && id[i] < a.E.v;
    const float sc = __uint_as_float((uint32_t)s[i] << 16);
    const float ze = __uint_as_float((uint32_t)z[i] << 16);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = in ? sc * (code_at(q[i], j) - ze) : 0.0f;
    uint8_t* out = a.out + (r0 + i) * a.o_bytes + (int64_t)col * sizeof(TO);
    if constexpr (sizeof(TO) == 2) {
      v8bf b;
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = (__bf16)y[j];
      *reinterpret_cast<v8bf*>(out) = b;
    } else {
      reinterpret_cast<v4f*>(out)[0] = v4f{y[0], y[1], y[2], y[3]};
      reinterpret_cast<v4f*>(out)[1] = v4f{y[4], y[5], y[6], y[7]};
    }
  }
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------
// The matrix instruction (16 rows of E by 16 rows of h by 32 columns) takes 8
// bf16 values a lane.  A code becomes one in two instructions for two columns:
// its 4 bits go to the upper 4 bits of the fraction of a bf16 number between 16
// and 32, where they count 1 each, and the code's sign bit is turned over, so
// that the number is 24 + q exactly.  The products with 24 are taken off by the
// sum of -h, a product of h with -1 that is the same for every row of E:
//   sum_k (q - zero) h = (24 + zero) sum_k (-h) + sum_k (24 + q) h.
// Both sums are fp32 sums of exact products, up to 24 sum |h| large on the way; but
// the matrix instruction rounds once for several products, so that the logits are about
// as near as those of a plain fp32 product, for an h of one sign as well (d = 2048, E of
// normal values: 0.7 to 1.9e-7 of their norm for mixed signs, a plain product 1.0 to
// 3.4e-7; bf16 h of one sign 1.1 to 4.6e-8 and 0.9 to 3.3e-8).

// The columns of a block of 128 that lane 16 q + . gives to product i: whole
// groups for the products of a group, and for groups of 128 one load of 16 bytes.
template <int kGroup>
__device__ __forceinline__ constexpr int column_of(int i, int q) {
  if (kGroup == 128) return 32 * q + 8 * i;
  if (kGroup == 64) return 64 * (i >> 1) + 16 * q + 8 * (i & 1);
  return 32 * i + 8 * q;
}

// Where chunk k (8 columns) of a block's 16 lies in a row of h in LDS, before the
// row's number is added to it (exclusively): with that, lanes of one chunk touch 16
// different slots.  The instruction that reads 16 bytes a lane takes lanes of two
// values of q at once, the one with c 0-3 and 12-15, the other with 4-11, whose
// chunks must not differ by 4: for groups of 128 they would, and a third of the reads
// waited.
template <int kGroup>
__device__ __forceinline__ constexpr int place_of_chunk(int k) {
  return kGroup == 128 ? (k & 1) | (k >> 1 & 6) | (k << 2 & 8) : k;
}

// A lane's codes of a block, of the row at byte `row` from p.
template <int kGroup>
__device__ __forceinline__ v4u load_codes(const uint8_t* p, uint32_t row, int q) {
  if constexpr (kGroup == 128) {
    return *reinterpret_cast<const v4u*>(p + (row + 16 * q));
  } else if constexpr (kGroup == 64) {
    const v2u a = *reinterpret_cast<const v2u*>(p + (row + 8 * q));
    const v2u b = *reinterpret_cast<const v2u*>(p + (row + 8 * q) + 32);
    return v4u{a.x, a.y, b.x, b.y};
  } else {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(p + (row + 4 * q) + 16 * i);
    return w;
  }
}
// The same of a block that ends after `left` columns: the block's first codes
// instead of those past its end (h is zero there).
template <int kGroup>
__device__ __forceinline__ v4u load_codes_cut(const uint8_t* p, uint32_t row, int q, int left) {
  v4u w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = column_of<kGroup>(i, q);
    w[i] = *reinterpret_cast<const uint32_t*>(p + (row + (c < left ? c / 2 : 0)));
  }
  return w;
}

// 24 + q of 8 columns
__device__ __forceinline__ v8bf unpack(uint32_t w) {
  const v4u x = {((w << 3) & 0x00780078u) ^ 0x41C041C0u, ((w >> 1) & 0x00780078u) ^ 0x41C041C0u,
                 ((w >> 5) & 0x00780078u) ^ 0x41C041C0u, ((w >> 9) & 0x00780078u) ^ 0x41C041C0u};
  return __builtin_bit_cast(v8bf, x);
}
__device__ __forceinline__ v8bf minus1() {
  const v4u x = {0xBF80BF80u, 0xBF80BF80u, 0xBF80BF80u, 0xBF80BF80u};
  return __builtin_bit_cast(v8bf, x);
}

// 8 columns of a row of h as bf16 numbers: itself, or an fp32 number's upper,
// middle and lower 8 bits, whose sum it is.  The products with the upper part
// and with the others are summed apart (kSums): the first sums hold few bits and
// are taken off again nearly without rounding, and the others are 2^-8 of them.
template <typename T>
struct RowOfH;
template <>
struct RowOfH<bf16_t> {
  static constexpr int kBytes = 2, kParts = 1, kSums = 1;
  v8bf x[1];
  __device__ __forceinline__ void load(const uint8_t* p) {
    x[0] = *reinterpret_cast<const v8bf*>(p);
  }
  __device__ __forceinline__ void clear() { x[0] = __builtin_bit_cast(v8bf, v4u{0, 0, 0, 0}); }
};
template <>
struct RowOfH<float> {
  static constexpr int kBytes = 4, kParts = 3, kSums = 2;
  v8bf x[3];
  __device__ __forceinline__ void split(float* y) {
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      v4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = __float_as_uint(y[2 * j]), b = __float_as_uint(y[2 * j + 1]);
        w[j] = __builtin_amdgcn_perm(b, a, 0x07060302);
        y[2 * j] -= __uint_as_float(a & 0xFFFF0000u);
        y[2 * j + 1] -= __uint_as_float(b & 0xFFFF0000u);
      }
      x[part] = __builtin_bit_cast(v8bf, w);
    }
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
    float y[8];
    load_whole8<float>(p, 0, y);
    split(y);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int part = 0; part < 3; ++part) x[part] = __builtin_bit_cast(v8bf, v4u{0, 0, 0, 0});
  }
};

// The sums of a 16 x 16 tile over a group.
template <typename T>
struct Sums {
  v4f x[RowOfH<T>::kSums];
  // += A . (8 columns of each row of h), the smallest parts first
  __device__ __forceinline__ void add(const v8bf& a, const RowOfH<T>& h) {
#pragma unroll
    for (int part = RowOfH<T>::kParts - 1; part >= 0; --part)
      x[part ? 1 : 0] =
          __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, h.x[part], x[part ? 1 : 0], 0, 0, 0);
  }
  // what the group adds to the logits: less = the sums of -h
  __device__ __forceinline__ v4f with_zero(v4f z, const Sums& less) const {
    Sums y = *this;
#pragma unroll
    for (int p = 0; p < RowOfH<T>::kSums; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) y.x[p][i] = fmaf(z[i], less.x[p][i], y.x[p][i]);
    return y.all();
  }
  __device__ __forceinline__ v4f all() const {
    if constexpr (RowOfH<T>::kSums == 1) return x[0];
    else return x[0] + x[1];
  }
};

// 4 neighbouring scales (or zeros); past the last token the last one's
__device__ __forceinline__ v2u load4(const uint16_t* p, int64_t t, int64_t v, bool whole) {
  if (whole) return *reinterpret_cast<const v2u*>(p + t);
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = p[t + i < v ? t + i : v - 1];
  return v2u{x[0] | x[1] << 16, x[2] | x[3] << 16};
}
__device__ __forceinline__ v4f spread4(v2u w) {
  return v4f{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}

__device__ __forceinline__ void store4(const LogitsInt4Args& a, int out_size, int m, int64_t t,
                                       v4f x) {
  if (out_size == 4) {
    float* row = reinterpret_cast<float*>(a.out) + (int64_t)m * a.ldo;
    if (t + 4 <= a.E.v) {
      *reinterpret_cast<v4f*>(row + t) = x;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i < a.E.v) row[t + i] = x[i];
    }
  } else {
    __bf16* row = reinterpret_cast<__bf16*>(a.out) + (int64_t)m * a.ldo;
    typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
    if (t + 4 <= a.E.v) {
      *reinterpret_cast<v4bf*>(row + t) = __builtin_convertvector(x, v4bf);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i < a.E.v) row[t + i] = (__bf16)x[i];
    }
  }
}

// 16 MT rows of h by 16 NT of E per workgroup, whose kSplit waves take every
// kSplit-th block of 128 columns and join their sums: for vocabularies with too few
// tiles, where a wave's chain of blocks sets the time (1 x 5003 x 1104 bf16 7.3 us, 12
// with tiles of 64 x 128; 9 rows in fp32 with groups of 32 and zeros 10.3, most of it the
// launch, two round trips to memory and the parts of h).
template <int MT, int NT, int kSplit, int kGroup, typename TH>
__global__ __launch_bounds__(64 * kSplit) void logits4_rows_kernel(const LogitsInt4Args a, int out_size) {
  constexpr int kSubs = 128 / kGroup, kEach = kGroup / 32;   // groups; products of one
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT;
  const int m0 = blockIdx.y * 16 * MT;
  const bool whole = n0 + 16 * NT <= a.E.v;
  const uint8_t* const e_base = a.E.codes + n0 * a.E.c_bytes;
  uint32_t e_row[NT];
  const uint8_t* h[MT];
  const int e_last = (int)min(a.E.v - 1 - n0, (int64_t)16 * NT);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    e_row[j] = (uint32_t)min(16 * j + c, e_last) * (uint32_t)a.E.c_bytes;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + c;
    h[t] = a.h + (int64_t)(m < a.rows ? m : a.rows - 1) * a.h_bytes;
  }
  v4f acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int blocks = (a.E.d + 127) / 128;
  v4u codes[NT];
  v2u scale[kSubs][NT], zero[kSubs][NT];
  auto load = [&](int kb) {
    const int left = a.E.d - kb * 128;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      codes[j] = left >= 128 ? load_codes<kGroup>(e_base + kb * 64, e_row[j], q)
                             : load_codes_cut<kGroup>(e_base + kb * 64, e_row[j], q, left);
#pragma unroll
    for (int s = 0; s < kSubs; ++s) {
      const int g = kb * kSubs + s < a.E.groups ? kb * kSubs + s : a.E.groups - 1;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        scale[s][j] = load4(a.E.scale + g * a.E.lds, n0 + 16 * j + 4 * q, a.E.v, whole);
        if (a.E.zero)
          zero[s][j] = load4(a.E.zero + g * a.E.lds, n0 + 16 * j + 4 * q, a.E.v, whole);
      }
    }
  };
  int kb = w;
  if (kb < blocks) load(kb);
  for (; kb < blocks; kb += kSplit) {
    RowOfH<TH> hf[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kb * 128 + column_of<kGroup>(i, q);
        if (k < a.E.d) hf[t][i].load(h[t] + k * RowOfH<TH>::kBytes);
        else hf[t][i].clear();
      }
    v4u now[NT];
    v2u s_now[kSubs][NT], z_now[kSubs][NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      now[j] = codes[j];
#pragma unroll
      for (int s = 0; s < kSubs; ++s) {
        s_now[s][j] = scale[s][j];
        z_now[s][j] = zero[s][j];
      }
    }
    if (kb + kSplit < blocks) load(kb + kSplit);
#pragma unroll
    for (int s = 0; s < kSubs; ++s) {
      Sums<TH> less[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int p = 0; p < RowOfH<TH>::kSums; ++p) less[t].x[p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int f = 0; f < kEach; ++f) less[t].add(minus1(), hf[t][s * kEach + f]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Sums<TH> x[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int p = 0; p < RowOfH<TH>::kSums; ++p) x[t].x[p] = less[t].x[p] * 24.0f;
#pragma unroll
        for (int f = 0; f < kEach; ++f) {
          const v8bf b = unpack(now[j][s * kEach + f]);
#pragma unroll
          for (int t = 0; t < MT; ++t) x[t].add(b, hf[t][s * kEach + f]);
        }
        const v4f sc = spread4(s_now[s][j]);
        const v4f z = a.E.zero ? spread4(z_now[s][j]) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const v4f y = a.E.zero ? x[t].with_zero(z, less[t]) : x[t].all();
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(y[i], sc[i], acc[t][j][i]);
        }
      }
    }
  }
  __shared__ v4f s_acc[(kSplit - 1) * MT * NT * 64];
  if (w > 0) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) s_acc[(((w - 1) * MT + t) * NT + j) * 64 + lane] = acc[t][j];
  }
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int u = 0; u < kSplit - 1; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[t][j] += s_acc[((u * MT + t) * NT + j) * 64 + lane];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + c;
    if (m < a.rows)
#pragma unroll
      for (int j = 0; j < NT; ++j) store4(a, out_size, m, n0 + 16 * j + 4 * q, acc[t][j]);
  }
}

// Tiles: kBM rows of h by kBN of E per workgroup of W waves, S blocks of 128
// columns at a time.  A wave reads the codes of its own rows of E into
// registers, a step ahead, so that every code is read and unpacked once; the rows of
// h go through LDS (two buffers), and with them the sums of -h, and the scales.
//
// Few rows are bound by memory: 1 x 128256 x 2048 takes 29 us for 135 MB (4.6 TB/s;
// three or eight such E in turn, more than the caches hold; 25 for two, which they hold
// in part) with two blocks at a time, which read whole lines of the codes, and 34 with
// one.
// For 64 rows and more the unpacking, the scales and the products take turns: 512 x
// 128256 x 2048 takes 309 to 317 us (0.87 PFLOP/s, the matrix units 35 % busy, four
// vector instructions for each of theirs; a library's product with E in bf16 271),
// 64 rows 50 (four tiles of E a wave; 61 with two).  With groups of 32 and zeros 512 rows
// take 645 (groups of 32 alone 610, of 64 with zeros 417): a product has its own scales
// then.  Reads of h from LDS a product ahead, wave priorities around the products, or
// codes read two steps ahead change 2 %.
// 40 x 262144 x 1152 with groups of 64 and zeros takes 62 (3.4 TB/s); zeros enter where
// a group's sums start (added at its end: 63.5, and 16 more registers).
template <int MT, int NT, int W, int S, int kWavesPerSimd, int kGroup, typename TH,
          bool kZero>
__global__ __launch_bounds__(64 * W, kWavesPerSimd) void logits4_tiles_kernel(
    const LogitsInt4Args a, int out_size) {
  constexpr int kSubs = 128 / kGroup, kEach = kGroup / 32, kLanes = kGroup / 8;
  constexpr int kThreads = 64 * W, kBM = 16 * MT, kBN = 16 * NT * W;
  constexpr int kParts = RowOfH<TH>::kParts, kSums = RowOfH<TH>::kSums;
  constexpr int kWords = RowOfH<TH>::kBytes / 2;    // 16-byte words of 8 columns of h
  constexpr int kRowChunks = 16 * S;                // of 8 columns, of a row of h
  constexpr int kChunks = (kBM * kRowChunks + kThreads - 1) / kThreads;   // a thread
  // chunk k of row r is in slot place(k) ^ (r & 15) of its block
  __shared__ __align__(16) v4u s_h[2][kParts][kBM * kRowChunks];
  __shared__ float s_less[2][kSums][S * kSubs][kBM];
  __shared__ __align__(16) float s_scale[2][S * kSubs][kBN], s_zero[2][S * kSubs][kZero ? kBN : 1];
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups are dealt to the 8 compute dies in turn: a die takes all tiles of
  // h under one of E one after the other, and reads its codes into its cache once.
  const unsigned mt = (unsigned)(a.rows + kBM - 1) / kBM;
  const unsigned local = blockIdx.x / 8;
  const int m0 = (int)(local % mt) * kBM;
  const int64_t n0 = ((int64_t)(local / mt) * 8 + blockIdx.x % 8) * kBN;
  if (n0 >= a.E.v) return;
  const int64_t nw = n0 + w * 16 * NT;       // the wave's rows of E
  // (32-bit offsets from the wave's first row)
  const uint8_t* const e_base = a.E.codes + (nw < a.E.v ? nw : a.E.v - 1) * a.E.c_bytes;
  const int e_last = (int)(nw < a.E.v ? min(a.E.v - 1 - nw, (int64_t)16 * NT) : 0);
  uint32_t e_row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    e_row[j] = (uint32_t)min(16 * j + c, e_last) * (uint32_t)a.E.c_bytes;
  const int blocks = (a.E.d + 127) / 128, steps = (blocks + S - 1) / S;
  struct Codes { v4u x[S][NT]; };
  // (past the last block the last one again, so that loads are counted alike)
  auto load_e = [&](int step) {
    Codes r;
#pragma unroll
    for (int b = 0; b < S; ++b) {
      const int kb = min(step * S + b, blocks - 1);
      const int left = a.E.d - kb * 128;
      const uint8_t* base = e_base + kb * 64;
      if (left >= 128) {
#pragma unroll
        for (int j = 0; j < NT; ++j) r.x[b][j] = load_codes<kGroup>(base, e_row[j], q);
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) r.x[b][j] = load_codes_cut<kGroup>(base, e_row[j], q, left);
      }
    }
    return r;
  };
  // scales of two neighbouring tokens: memory to registers, and those to LDS as
  // fp32 numbers
  constexpr int kPairs = kBN / 2 * kSubs * S, kEachS = (kPairs + kThreads - 1) / kThreads;
  struct Scales { uint32_t s[kEachS], z[kEachS]; };
  auto load_s = [&](int step) {
    Scales r;
#pragma unroll
    for (int i = 0; i < kEachS; ++i) {
      const int id = i * kThreads + tid, sub = id / (kBN / 2), pair = id % (kBN / 2) * 2;
      r.s[i] = r.z[i] = 0u;
      if (kPairs % kThreads == 0 || id < kPairs) {
        const int g = min(step * S * kSubs + sub, a.E.groups - 1);
        const int64_t t = n0 + pair;
        const bool two = t + 1 < a.E.v;
        const int64_t at = g * a.E.lds + (two ? t : a.E.v - 1);
        r.s[i] = two ? *reinterpret_cast<const uint32_t*>(a.E.scale + at) : a.E.scale[at];
        if constexpr (kZero)
          r.z[i] = two ? *reinterpret_cast<const uint32_t*>(a.E.zero + at) : a.E.zero[at];
      }
    }
    return r;
  };
  auto store_s = [&](Scales r, int step) {
#pragma unroll
    for (int i = 0; i < kEachS; ++i) {
      const int id = i * kThreads + tid, sub = id / (kBN / 2), pair = id % (kBN / 2) * 2;
      if (kPairs % kThreads == 0 || id < kPairs) {
        *reinterpret_cast<float2*>(&s_scale[step & 1][sub][pair]) =
            make_float2(bf16_lo(r.s[i]), bf16_hi(r.s[i]));
        if constexpr (kZero)
          *reinterpret_cast<float2*>(&s_zero[step & 1][sub][pair]) =
              make_float2(24.0f + bf16_lo(r.z[i]), 24.0f + bf16_hi(r.z[i]));
      }
    }
  };
  // rows of h: memory to registers, and those to LDS
  struct Raw { v4u x[kChunks][kWords]; };
  const int u = tid % kRowChunks;
  const uint8_t* const h_base = a.h + (int64_t)m0 * a.h_bytes;
  uint32_t h_row[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    h_row[i] =
        (uint32_t)min((i * kThreads + tid) / kRowChunks, a.rows - 1 - m0) * (uint32_t)a.h_bytes;
  auto load_h = [&](int step) {
    step = min(step, steps - 1);
    // (a chunk past the row's end: the step's first one; it is cleared below)
    const uint8_t* base = h_base + step * S * 128 * RowOfH<TH>::kBytes;
    const uint32_t k = step * S * 128 + u * 8 < a.E.d ? u * 8 * RowOfH<TH>::kBytes : 0;
    Raw r;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        r.x[i][j] = *reinterpret_cast<const v4u*>(base + (h_row[i] + k) + 16 * j);
    return r;
  };
  auto store_h = [&](Raw r, int step) {
    const int buf = step & 1;
    const bool in = step * S * 128 + u * 8 < a.E.d;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + tid, row = id / kRowChunks;
      if (kBM * kRowChunks % kThreads && id >= kBM * kRowChunks) break;
      RowOfH<TH> h;
      float less[kSums];
      if constexpr (kParts == 1) {
        h.x[0] = __builtin_bit_cast(v8bf, in ? r.x[i][0] : v4u{0, 0, 0, 0});
        const v4u b = __builtin_bit_cast(v4u, h.x[0]);
        const float minus = __uint_as_float(0xBF80BF80u);   // two of -1
        less[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) less[0] = dot2_bf16(b[j], minus, less[0]);
      } else {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = in ? __uint_as_float(r.x[i][j / 4][j % 4]) : 0.0f;
        less[0] = less[kSums - 1] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float upper = __uint_as_float(__float_as_uint(y[j]) & 0xFFFF0000u);
          less[0] -= upper;
          less[kSums - 1] -= y[j] - upper;
        }
        h.split(y);
      }
#pragma unroll
      for (int p = 0; p < kParts; ++p)
        s_h[buf][p][row * kRowChunks + (u & ~15) + (place_of_chunk<kGroup>(u & 15) ^ (row & 15))] =
            __builtin_bit_cast(v4u, h.x[p]);
#pragma unroll
      for (int p = 0; p < kSums; ++p) {
        const float sum = group_sum<kLanes>(less[p]);
        if (u % kLanes == 0) s_less[buf][p][u / kLanes][row] = sum;
      }
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  Raw raw = load_h(0);
  Scales sc = load_s(0);
  Codes next = load_e(0);
  store_h(raw, 0);
  store_s(sc, 0);
  raw = load_h(1);
  sc = load_s(1);
  __syncthreads();
  for (int step = 0; step < steps; ++step) {
    const Codes now = next;
    next = load_e(step + 1);
    const int buf = step & 1;
    Sums<TH> x[MT][NT];
    v4f scale[NT];
#pragma unroll
    for (int i = 0; i < S * 4; ++i) {   // products
      const int b = i / 4, sub = i / kEach;   // block of the step, group of the step
      if (S > 1 && i % 4 == 0 && b > 0 && step * S + b >= blocks) break;
      if (i % kEach == 0) {
        // the group's sums start at (24 + z) (-h)
        float less[MT][kSums];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int p = 0; p < kSums; ++p) less[t][p] = s_less[buf][p][sub][t * 16 + c];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          v4f by = v4f{24.0f, 24.0f, 24.0f, 24.0f};
          if constexpr (kZero)
            by = *reinterpret_cast<const v4f*>(&s_zero[buf][sub][(w * NT + j) * 16 + 4 * q]);
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int p = 0; p < kSums; ++p) x[t][j].x[p] = by * less[t][p];
        }
      }
      const int slot = 16 * b + (place_of_chunk<kGroup>(column_of<kGroup>(i % 4, q) / 8) ^ c);
      RowOfH<TH> h[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          h[t].x[p] = __builtin_bit_cast(
              v8bf, s_h[buf][p][(t * 16 + c) * kRowChunks + slot]);
      const bool last = i % kEach == kEach - 1;
      if (last) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int n = (w * NT + j) * 16 + 4 * q;
          scale[j] = *reinterpret_cast<const v4f*>(&s_scale[buf][sub][n]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // (more in flight does not fit the registers)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v8bf e = unpack(now.x[b][j][i % 4]);
#pragma unroll
        for (int t = 0; t < MT; ++t) x[t][j].add(e, h[t]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (!last) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const v4f y = x[t][j].all();
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][j][r] = fmaf(y[r], scale[j][r], acc[t][j][r]);
          asm volatile("" : "+v"(acc[t][j]));   // (the sums here, not at the step's end)
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (step + 1 < steps) {
      store_h(raw, step + 1);
      store_s(sc, step + 1);
      raw = load_h(step + 2);
      sc = load_s(step + 2);
      __syncthreads();
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + t * 16 + c;
    if (m < a.rows)
#pragma unroll
      for (int j = 0; j < NT; ++j) store4(a, out_size, m, nw + 16 * j + 4 * q, acc[t][j]);
  }
}

template <int MT, int NT, int W, int S, int kWavesPerSimd, int kGroup, typename TH>
void enqueue_tiles(const LogitsInt4Args& a, int out_size, hipStream_t s) {
  constexpr int kBM = 16 * MT, kBN = 16 * NT * W;
  const int64_t mt = (a.rows + kBM - 1) / kBM, nt = (a.E.v + kBN - 1) / kBN;
  const dim3 grid((unsigned)(8 * ((nt + 7) / 8) * mt)), block(64 * W);
  if (a.E.zero)
    hipLaunchKernelGGL((logits4_tiles_kernel<MT, NT, W, S, kWavesPerSimd, kGroup, TH, true>),
                       grid, block, 0, s, a, out_size);
  else
    hipLaunchKernelGGL((logits4_tiles_kernel<MT, NT, W, S, kWavesPerSimd, kGroup, TH, false>),
                       grid, block, 0, s, a, out_size);
}

template <int MT, int NT, int kSplit, int kGroup, typename TH>
void enqueue_rows(const LogitsInt4Args& a, int out_size, hipStream_t s) {
  hipLaunchKernelGGL((logits4_rows_kernel<MT, NT, kSplit, kGroup, TH>),
                     dim3((unsigned)((a.E.v + 16 * NT - 1) / (16 * NT)),
                          (unsigned)((a.rows + 16 * MT - 1) / (16 * MT))),
                     dim3(64 * kSplit), 0, s, a, out_size);
}

template <int kGroup, typename TH>
void enqueue_logits(const LogitsInt4Args& a, int out_size, hipStream_t s) {
  constexpr bool kF32 = RowOfH<TH>::kParts == 3;
  switch (plan_logits4(a.rows, a.E.v, kF32)) {
    case Logits4Plan::kRows16: enqueue_rows<1, 2, 8, kGroup, TH>(a, out_size, s); break;
    case Logits4Plan::kRows32: enqueue_rows<2, 2, 4, kGroup, TH>(a, out_size, s); break;
    case Logits4Plan::k16x128:
      enqueue_tiles<1, 2, 4, kF32 ? 1 : 2, 4, kGroup, TH>(a, out_size, s);
      break;
    case Logits4Plan::k32x256:
      enqueue_tiles<2, 4, 4, kF32 ? 1 : 2, 2, kGroup, TH>(a, out_size, s);
      break;
    case Logits4Plan::k48x256:
      if constexpr (!kF32) enqueue_tiles<3, 4, 4, 1, 2, kGroup, TH>(a, out_size, s);
      break;
    case Logits4Plan::k64x128:
      if constexpr (!kF32) enqueue_tiles<4, 2, 4, 1, 2, kGroup, TH>(a, out_size, s);
      break;
    case Logits4Plan::k64x256:
      if constexpr (kF32) enqueue_tiles<4, 2, 8, 1, 2, kGroup, TH>(a, out_size, s);
      break;
    case Logits4Plan::k64x512:
      if constexpr (!kF32) enqueue_tiles<4, 4, 8, 1, 2, kGroup, TH>(a, out_size, s);
      break;
  }
}

}  // namespace

hipError_t launch_quantize_int4(const QuantizeInt4Args& a, int dtype, hipStream_t s) {
  const bool bf16 = dtype == FH_DTYPE_BF16;
  switch (a.group) {
    case 32: bf16 ? enqueue_quantize<uint16_t, 32>(a, s) : enqueue_quantize<float, 32>(a, s); break;
    case 64: bf16 ? enqueue_quantize<uint16_t, 64>(a, s) : enqueue_quantize<float, 64>(a, s); break;
    default: bf16 ? enqueue_quantize<uint16_t, 128>(a, s) : enqueue_quantize<float, 128>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_int4_rows(const Int4RowsArgs& a, int group, int out_dtype, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 4 * kReadRows - 1) / (4 * kReadRows) *
                             ((a.E.d + 511) / 512)));
  const int shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  auto enqueue = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, shift);
  };
  if (out_dtype == FH_DTYPE_BF16)
    a.E.zero ? enqueue(int4_rows_kernel<uint16_t, true>)
             : enqueue(int4_rows_kernel<uint16_t, false>);
  else
    a.E.zero ? enqueue(int4_rows_kernel<float, true>) : enqueue(int4_rows_kernel<float, false>);
  return hipGetLastError();
}

hipError_t launch_logits_int4(const LogitsInt4Args& a, int group, int h_dtype, int out_dtype,
                              hipStream_t s) {
  const bool bf16 = h_dtype == FH_DTYPE_BF16;
  const int size = out_dtype == FH_DTYPE_BF16 ? 2 : 4;
  switch (group) {
    case 32:
      bf16 ? enqueue_logits<32, bf16_t>(a, size, s) : enqueue_logits<32, float>(a, size, s);
      break;
    case 64:
      bf16 ? enqueue_logits<64, bf16_t>(a, size, s) : enqueue_logits<64, float>(a, size, s);
      break;
    default:
      bf16 ? enqueue_logits<128, bf16_t>(a, size, s) : enqueue_logits<128, float>(a, size, s);
  }
  return hipGetLastError();
}

}  // namespace fh
