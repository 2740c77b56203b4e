// Host-only parts of libflashhead: the checks flashhead_prepare makes of its
// descriptor (the cluster table C2T among them) and the INT4 centroid
// quantizer of the FlashHead reading notes (Module 3, selective quantization).
// Nothing here touches a device or a HIP type, so the same source also builds
// with a plain host compiler, as the sanitizer test on the CPU does.
#pragma once

#include <stdint.h>

#include <vector>

#include "../../include/flashhead.h"

namespace fh {

int esize_of(int dtype);  // bytes per element of an FH_DTYPE_*, 0 if unknown
bool aligned16(const void* p);

// FH_OK, or the status flashhead_prepare returns for this descriptor before
// it touches the device: FH_ERR_INVALID_ARG, FH_ERR_UNSUPPORTED or
// FH_ERR_NOT_PERMUTATION.  Reads ds->c2t (host memory, v entries).
int validate_desc(const fh_desc* ds);

// FH_OK when t[0..v) holds every value of [0, v) once (equal-size clusters in
// a dense c x b table: FlashHead reading notes, Module 1), else
// FH_ERR_NOT_PERMUTATION.
int check_permutation(const int32_t* t, int64_t v);

// inv[t[r]] = r for a permutation t of [0, v): the row of each token in the
// cluster-major layout.
void invert_permutation(const int32_t* t, int64_t v, int32_t* inv);

double round_bf16(double x);     // nearest bf16 value, ties to even
uint16_t bf16_bits(double x);    // bits of a value that is already a bf16 value
double bf16_value(uint16_t bits);

// bf16 of each column's mean over the c rows of C (c x d, bf16 bits): the
// shift of the mean-shifted INT4 variant.
void column_mean_shift(const uint16_t* C, int c, int d, std::vector<double>& mu);

// Symmetric INT4 codes per group of 128 columns of C - shift (shift: d values,
// or null): scale = bf16(amax / 7), code = round-half-even(x / scale) clipped
// to [-8, 7].  Codes are packed in tiles of 16 centroid rows: for tile t and
// group g, 64 lanes of 16 bytes, lane = quarter * 16 + row-in-tile, byte j of
// a lane holding columns quarter * 32 + 2j (low nibble) and + 1 (high nibble).
// Scales: [tile][group][row-in-tile] bf16 bits.  d must be a multiple of 128;
// rows past c in the last tile are left zero.
void quantize_int4(const uint16_t* C, const double* shift, int c, int d,
                   std::vector<uint8_t>& codes, std::vector<uint16_t>& scales, int* ntiles_out,
                   int* groups_out);

// The kernel of a dense_logits_fp8 call: tiles of bm rows of h by bn of E, which
// kLogits8Groups workgroups take one after the other, or (few rows, or few
// tiles) a workgroup for every bm x bn, whose kLogits8Split waves share d.
constexpr int kLogits8Groups = 256;  // compute units
constexpr int kLogits8Split = 4;
struct Logits8Plan {
  bool tiles;
  int bm, bn;
};
Logits8Plan plan_logits8(int64_t rows, int64_t v, int32_t d, int64_t ldo, int out_size);

// The row stride that a call uses of an optional matrix: 0 where no second row
// is there (such a stride may hold anything).
int64_t row_stride(const void* p, int64_t ld, int64_t rows);

// The argument checks of the calls around the 8-bit head (see
// include/flashhead.h for what each call accepts): FH_OK, or the status the
// call returns before it touches the device.
int check_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                  const void* weight, int64_t rows, int32_t d, int32_t dtype, float eps,
                  float weight_offset, const void* residual_out, int64_t ldro, const void* y,
                  int64_t ldy, const void* y8, int64_t ldy8, const void* y_scale, int64_t lds);
int check_quantize_fp8(const void* E, int64_t v, int32_t d, int32_t dtype, int64_t lde,
                       const void* E8, int64_t lde8, const void* E_scale, int64_t lds);
int check_logits_fp8(const void* h8, int64_t ldh, const void* h_scale, int64_t lds, int32_t rows,
                     const void* E8, int64_t lde, const void* E_scale, int64_t ldes, int64_t v,
                     int32_t d, const void* out, int32_t out_dtype, int64_t ldo);
bool verify_fits(int64_t rows, int32_t B, int64_t v);  // v in [1, 2^31)
int check_verify(const void* logits, int64_t rows, int64_t v, int32_t dtype, int64_t ldl,
                 const void* row_start, int32_t B, const void* draft_tokens, int64_t n_drafts,
                 const void* draft_probs, int64_t ldq, int32_t mode, float tau,
                 const void* u_accept, const void* u_sample, int32_t max_tokens,
                 const void* out_tokens, const void* out_accepted, const void* workspace);

}  // namespace fh
