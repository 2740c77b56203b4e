// Host-only checks, the INT4 centroid quantizer and the choice of the 8-bit
// logits' kernel (declarations and their contracts in fh_host.h).
#include "fh_host.h"

#include <math.h>
#include <string.h>

namespace fh {

int esize_of(int dtype) { return dtype == FH_DTYPE_F32 ? 4 : dtype == FH_DTYPE_BF16 ? 2 : 0; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check_permutation(const int32_t* t, int64_t v) {
  if (!t || v < 1) return FH_ERR_NOT_PERMUTATION;
  std::vector<uint8_t> seen((size_t)v, 0);
  for (int64_t i = 0; i < v; ++i) {
    const int32_t x = t[i];
    if (x < 0 || (int64_t)x >= v || seen[(size_t)x]) return FH_ERR_NOT_PERMUTATION;
    seen[(size_t)x] = 1;
  }
  return FH_OK;
}

void invert_permutation(const int32_t* t, int64_t v, int32_t* inv) {
  for (int64_t r = 0; r < v; ++r) inv[(size_t)t[r]] = (int32_t)r;
}

int validate_desc(const fh_desc* ds) {
  if (!ds || !ds->E || !ds->c2t) return FH_ERR_INVALID_ARG;
  if (ds->c < 1 || ds->b < 1 || ds->d < 1 || ds->v != (int64_t)ds->c * ds->b)
    return FH_ERR_INVALID_ARG;
  if (ds->max_batch < 1 || ds->max_batch > FH_MAX_BATCH) return FH_ERR_INVALID_ARG;
  if (ds->max_p < 1 || ds->max_p > ds->c) return FH_ERR_INVALID_ARG;
  if (ds->lde < ds->d) return FH_ERR_INVALID_ARG;
  if (ds->v > (int64_t)INT32_MAX) return FH_ERR_UNSUPPORTED;
  const int es = esize_of(ds->dtype);
  if (!es) return FH_ERR_UNSUPPORTED;
  if (ds->c > FH_MAX_C) return FH_ERR_UNSUPPORTED;
  const int64_t row_bytes = (int64_t)ds->d * es;
  if (row_bytes % 16 || (ds->lde * es) % 16 || row_bytes > FH_MAX_ROW_BYTES)
    return FH_ERR_UNSUPPORTED;
  if (!aligned16(ds->E) || (ds->C && !aligned16(ds->C))) return FH_ERR_UNSUPPORTED;
  if (ds->quant != FH_QUANT_NONE && ds->quant != FH_QUANT_INT4_G128 &&
      ds->quant != FH_QUANT_INT4_G128_MEAN)
    return FH_ERR_UNSUPPORTED;
  if (ds->quant != FH_QUANT_NONE && (ds->dtype != FH_DTYPE_BF16 || ds->d % 128))
    return FH_ERR_UNSUPPORTED;
  if (ds->flags & ~(FH_FLAG_COOPERATIVE | FH_FLAG_BORROW_E | FH_FLAG_STREAM_ALL |
                    FH_FLAG_SELECT_FIRST))
    return FH_ERR_INVALID_ARG;
  if ((ds->flags & FH_FLAG_STREAM_ALL) && (ds->flags & FH_FLAG_SELECT_FIRST))
    return FH_ERR_INVALID_ARG;
  return check_permutation(ds->c2t, ds->v);
}

double round_bf16(double x) {
  if (x == 0.0 || !isfinite(x)) return x;
  int e = 0;
  (void)frexp(x, &e);
  // 8 significant bits; below the smallest normal exponent the spacing stays 2^-133
  const int se = (e - 8) > -133 ? (e - 8) : -133;
  return ldexp(nearbyint(ldexp(x, -se)), se);
}

uint16_t bf16_bits(double x) {
  const float f = (float)x;
  uint32_t u;
  memcpy(&u, &f, 4);
  return (uint16_t)(u >> 16);
}

double bf16_value(uint16_t b) {
  const uint32_t u = (uint32_t)b << 16;
  float f;
  memcpy(&f, &u, 4);
  return (double)f;
}

void column_mean_shift(const uint16_t* C, int c, int d, std::vector<double>& mu) {
  // the sum of c bf16 values is exact in double for the c the library accepts
  mu.assign((size_t)d, 0.0);
  for (int k = 0; k < c; ++k)
    for (int j = 0; j < d; ++j) mu[(size_t)j] += bf16_value(C[(size_t)k * d + j]);
  for (int j = 0; j < d; ++j) mu[(size_t)j] = round_bf16(mu[(size_t)j] / c);
}

void quantize_int4(const uint16_t* C, const double* shift, int c, int d,
                   std::vector<uint8_t>& codes, std::vector<uint16_t>& scales, int* ntiles_out,
                   int* groups_out) {
  const int G = d / 128, ntiles = (c + 15) / 16;
  codes.assign((size_t)ntiles * G * 1024, 0);
  scales.assign((size_t)ntiles * G * 16, 0);
  int8_t q[128];
  double x[128];
  for (int k = 0; k < c; ++k) {
    const int t = k / 16, rin = k % 16;
    for (int g = 0; g < G; ++g) {
      const uint16_t* src = C + (size_t)k * d + (size_t)g * 128;
      const double* sh = shift ? shift + (size_t)g * 128 : nullptr;
      double amax = 0.0;
      for (int j = 0; j < 128; ++j) {
        // x - shift is exact in double for bf16 x and shift
        x[j] = bf16_value(src[j]) - (sh ? sh[j] : 0.0);
        amax = fmax(amax, fabs(x[j]));
      }
      const double s = round_bf16(amax / 7.0);
      for (int j = 0; j < 128; ++j) {
        double qq = s > 0.0 ? nearbyint(x[j] / s) : 0.0;
        qq = qq < -8.0 ? -8.0 : (qq > 7.0 ? 7.0 : qq);
        q[j] = (int8_t)qq;
      }
      scales[((size_t)t * G + g) * 16 + rin] = bf16_bits(s);
      for (int quarter = 0; quarter < 4; ++quarter) {
        const int lane = quarter * 16 + rin;
        uint8_t* dst = codes.data() + (((size_t)t * G + g) * 64 + lane) * 16;
        for (int j = 0; j < 16; ++j) {
          const int col = quarter * 32 + 2 * j;
          dst[j] = (uint8_t)((q[col] & 0xF) | ((q[col + 1] & 0xF) << 4));
        }
      }
    }
  }
  *ntiles_out = ntiles;
  *groups_out = G;
}

namespace {

// one launch holds fewer than 2^32 threads, 256 of them a workgroup
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// rows `ld` elements of `es` bytes apart that no address space holds
bool too_far(int64_t ld, int es, int64_t rows) { return rows > 1 && ld > INT64_MAX / es / rows; }

// an optional matrix of `es`-byte elements whose rows start at multiples of 16 bytes
int check_rows16(const void* p, int64_t ld, int64_t cols, int es, int64_t rows) {
  if (!p) return FH_OK;
  if (rows > 1 && ld < cols) return FH_ERR_INVALID_ARG;
  if (!aligned16(p) || (rows > 1 && ld % (16 / es)) || too_far(ld, es, rows))
    return FH_ERR_UNSUPPORTED;
  return FH_OK;
}

}  // namespace

int64_t row_stride(const void* p, int64_t ld, int64_t rows) { return p && rows > 1 ? ld : 0; }

int check_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                  const void* weight, int64_t rows, int32_t d, int32_t dtype, float eps,
                  float weight_offset, const void* residual_out, int64_t ldro, const void* y,
                  int64_t ldy, const void* y8, int64_t ldy8, const void* y_scale, int64_t lds) {
  if (rows < 0 || d < 1 || !isfinite(eps) || eps < 0.0f || !isfinite(weight_offset))
    return FH_ERR_INVALID_ARG;
  if (rows > 0 && !x) return FH_ERR_INVALID_ARG;
  if (rows > 0 && !y && !y8 && !residual_out) return FH_ERR_INVALID_ARG;
  if ((y8 != nullptr) != (y_scale != nullptr)) return FH_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!es || d > FH_MAX_NORM_D || ((int64_t)d * es) % 16 || rows > kMaxGroups)
    return FH_ERR_UNSUPPORTED;
  if (weight && !aligned16(weight)) return FH_ERR_UNSUPPORTED;
  int st = check_rows16(x, ldx, d, es, rows);
  if (st == FH_OK) st = check_rows16(residual, ldr, d, es, rows);
  if (st == FH_OK) st = check_rows16(residual_out, ldro, d, es, rows);
  if (st == FH_OK) st = check_rows16(y, ldy, d, es, rows);
  if (st != FH_OK) return st;
  if (y8) {
    const int n = 16 / es;  // codes a thread stores at once
    if (rows > 1 && (ldy8 < d || lds < (d + 127) / 128)) return FH_ERR_INVALID_ARG;
    if (!aligned(y8, (uintptr_t)n) || (rows > 1 && ldy8 % n) || !aligned(y_scale, 4) ||
        too_far(ldy8, 1, rows) || too_far(lds, 4, rows))
      return FH_ERR_UNSUPPORTED;
  }
  return FH_OK;
}

int check_quantize_fp8(const void* E, int64_t v, int32_t d, int32_t dtype, int64_t lde,
                       const void* E8, int64_t lde8, const void* E_scale, int64_t lds) {
  if (!E || !E8 || !E_scale || v < 1 || d < 1) return FH_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!es || ((int64_t)d * es) % 16 || v > (int64_t)65535 * 128) return FH_ERR_UNSUPPORTED;
  const int st = check_rows16(E, lde, d, es, v);
  if (st != FH_OK) return st;
  if (v > 1 && lde8 < d) return FH_ERR_INVALID_ARG;
  if (v > 128 && lds < (d + 127) / 128) return FH_ERR_INVALID_ARG;
  const int n = 16 / es;
  if (!aligned(E8, (uintptr_t)n) || (v > 1 && lde8 % n) || !aligned(E_scale, 4) ||
      too_far(lde8, 1, v) || too_far(lds, 4, (v + 127) / 128))
    return FH_ERR_UNSUPPORTED;
  return FH_OK;
}

int check_logits_fp8(const void* h8, int64_t ldh, const void* h_scale, int64_t lds, int32_t rows,
                     const void* E8, int64_t lde, const void* E_scale, int64_t ldes, int64_t v,
                     int32_t d, const void* out, int32_t out_dtype, int64_t ldo) {
  if (rows < 0 || v < 1 || d < 1 || !E8 || !E_scale) return FH_ERR_INVALID_ARG;
  if (rows > 0 && (!h8 || !h_scale || !out)) return FH_ERR_INVALID_ARG;
  if (v > (int64_t)1 << 28 || rows > 65535 * 16) return FH_ERR_UNSUPPORTED;
  const int es = esize_of(out_dtype);
  if (!es || d % 16) return FH_ERR_UNSUPPORTED;
  const int32_t groups = (d + 127) / 128;
  if ((rows > 1 && lds < groups) || (v > 128 && ldes < groups)) return FH_ERR_INVALID_ARG;
  int st = check_rows16(h8, ldh, d, 1, rows);
  if (st == FH_OK) st = check_rows16(E8, lde, d, 1, v);
  if (st == FH_OK) st = check_rows16(out, ldo, v, es, rows);
  if (st != FH_OK) return st;
  if (!aligned(h_scale, 4) || !aligned(E_scale, 4)) return FH_ERR_UNSUPPORTED;
  // a tile's 256 rows are reached by 32-bit offsets
  const int64_t far = (int64_t)1 << 22;
  if ((rows > 1 && (ldh >= far || lds >= far)) || (v > 1 && lde >= far) ||
      (v > 128 && ldes >= far))
    return FH_ERR_UNSUPPORTED;
  return FH_OK;
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

Logits8Plan plan_logits8(int64_t rows, int64_t v, int32_t d, int64_t ldo, int out_size) {
  if (rows <= 16) {
    // As many rows of E a workgroup as leave most compute units one (1 x 4000
    // x 4096: 7 us with 16, 9 with 32; 16 x 32000 x 2048: 14 us with 64, 21
    // with 16); one row of h gains nothing from more than 32.
    if (v > 64 * 192 && rows > 4) return {false, 16, 64};
    return {false, 16, v > 32 * 192 ? 32 : 16};
  }
  // Estimated times in us.  Four waves with 32 rows of h and 64 of E, two
  // workgroups a compute unit: 2 us, 2.2 us for four blocks of columns, and E
  // once at the memory's rate (for 672 x 1424 x 560: 6 us, 8 with the smallest
  // tiles).
  const int64_t blocks = ceil_div(d, 128);
  Logits8Plan plan{false, 32, 64};
  double best = 2.0 +
                2.2 * (double)(ceil_div(ceil_div(rows, 32) * ceil_div(v, 64), 2 * kLogits8Groups) *
                               ceil_div(blocks, kLogits8Split)) +
                (double)v * d / 5.4e6;
  // Tiles: 3 us, and for each round of workgroups and each block the measured
  // time of a block (333 x 5003 x 1104, 64 x 16000 x 2048 and 40 x 20000 x 1024
  // with each tile; a smaller tile has more workgroups and less to do in each).
  static const struct {
    int bm, bn;
    double block;
  } kTiles[] = {{64, 128, 0.86}, {128, 128, 1.24}, {64, 256, 1.31}, {128, 256, 1.81}};
  // (the tiles reach 128 rows of out by 31-bit offsets)
  if (ldo * out_size < 1 << 23)
    for (const auto& t : kTiles) {
      const int64_t rounds =
          ceil_div(ceil_div(rows, t.bm) * ceil_div(v, t.bn), kLogits8Groups);
      const double time = 3.0 + (double)(rounds * blocks) * t.block;
      if (time < best) {
        best = time;
        plan = Logits8Plan{true, t.bm, t.bn};
      }
    }
  return plan;
}

bool verify_fits(int64_t rows, int32_t B, int64_t v) {
  // chunks of 2048 values; 512 threads a sequence
  const int64_t chunks = (v + 2047) / 2048;
  return rows <= kMaxGroups / chunks && B <= kMaxGroups / chunks && B <= kMaxGroups / 2;
}

int check_verify(const void* logits, int64_t rows, int64_t v, int32_t dtype, int64_t ldl,
                 const void* row_start, int32_t B, const void* draft_tokens, int64_t n_drafts,
                 const void* draft_probs, int64_t ldq, int32_t mode, float tau,
                 const void* u_accept, const void* u_sample, int32_t max_tokens,
                 const void* out_tokens, const void* out_accepted, const void* workspace) {
  if (B < 0 || rows < 0 || v < 1 || n_drafts < 0 || max_tokens < 1) return FH_ERR_INVALID_ARG;
  if (mode != FH_MODE_GREEDY && mode != FH_MODE_SAMPLE) return FH_ERR_INVALID_ARG;
  const bool sample = mode == FH_MODE_SAMPLE;
  if (sample && (!(tau > 0.0f) || !isfinite(tau))) return FH_ERR_INVALID_ARG;
  if (B > 0) {
    if (!row_start || !out_tokens || !out_accepted || !workspace) return FH_ERR_INVALID_ARG;
    if (rows > 0 && !logits) return FH_ERR_INVALID_ARG;
    if (n_drafts > 0 && (!draft_tokens || (sample && !u_accept))) return FH_ERR_INVALID_ARG;
    if (sample && !u_sample) return FH_ERR_INVALID_ARG;
  }
  if (draft_probs && !sample) return FH_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!es || v > (int64_t)INT32_MAX) return FH_ERR_UNSUPPORTED;
  int st = check_rows16(logits, ldl, v, es, rows);
  if (st == FH_OK) st = check_rows16(draft_probs, ldq, v, 4, n_drafts);
  if (st != FH_OK) return st;
  if (!aligned16(workspace)) return FH_ERR_UNSUPPORTED;
  return verify_fits(rows, B, v) ? FH_OK : FH_ERR_UNSUPPORTED;
}

}  // namespace fh
