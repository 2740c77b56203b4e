// CPU checks of the argument checks of the calls around the head (fh_host.cpp),
// built with the address and undefined-behaviour sanitizers by
// tests/test_around_sanitize.py: every argument at its ends, among them strides
// that no memory has.  Prints "ok <n>" with the number of checks and exits 0,
// or names the first failure and exits 1.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../two_stage_retrieval_amd/csrc/fh_host.h"

static int g_checks = 0;

#define CHECK(cond)                                                       \
  do {                                                                    \
    ++g_checks;                                                           \
    if (!(cond)) {                                                        \
      fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);   \
      exit(1);                                                            \
    }                                                                     \
  } while (0)

using namespace fh;

static void* const P = (void*)0x10000;  // aligned, never read
static const int64_t kEnds[] = {INT64_MIN,     INT64_MIN + 1,   -((int64_t)1 << 62), -1, 0, 1, 8, 255,
                                256,           264,             (int64_t)1 << 31,
                                (int64_t)1 << 60, ((int64_t)1 << 60) + 8, ((int64_t)1 << 61) + 8,
                                ((int64_t)1 << 62) + 8, INT64_MAX - 15, INT64_MAX};
static const int32_t kEnds32[] = {INT32_MIN, -1, 0, 1, 8, 16, 255, 256, 8192, 8200, INT32_MAX};

struct Norm {
  int64_t ldx = 256, ldr = 256, ldro = 256, ldy = 256, ldy8 = 256, lds = 2, rows = 4;
  int32_t d = 256, dtype = FH_DTYPE_BF16;
  float eps = 1e-6f, off = 0.0f;
  int operator()() const {
    return check_rmsnorm(P, ldx, P, ldr, P, rows, d, dtype, eps, off, P, ldro, P, ldy, P, ldy8, P,
                         lds);
  }
};
struct Quantize {
  int64_t v = 300, lde = 256, lde8 = 256, lds = 2;
  int32_t d = 256, dtype = FH_DTYPE_BF16;
  int operator()() const { return check_quantize_fp8(P, v, d, dtype, lde, P, lde8, P, lds); }
};
struct Logits {
  int64_t ldh = 256, lds = 2, lde = 256, ldes = 2, v = 300, ldo = 304;
  int32_t rows = 4, d = 256, dtype = FH_DTYPE_BF16;
  int operator()() const {
    return check_logits_fp8(P, ldh, P, lds, rows, P, lde, P, ldes, v, d, P, dtype, ldo);
  }
};
struct Verify {
  int64_t rows = 12, v = 1000, ldl = 1000, n = 8, ldq = 1000;
  int32_t B = 4, dtype = FH_DTYPE_BF16, mode = FH_MODE_SAMPLE, m = 3;
  float tau = 1.0f;
  int operator()() const {
    return check_verify(P, rows, v, dtype, ldl, P, B, P, n, P, ldq, mode, tau, P, P, m, P, P, P);
  }
};

// each 64-bit (32-bit) argument at every end, the others as they are, in both types
template <typename C>
static void ends64(int64_t C::*arg) {
  for (int t : {FH_DTYPE_BF16, FH_DTYPE_F32, 9})
    for (int64_t x : kEnds) {
      C c;
      c.dtype = t;
      c.*arg = x;
      const int st = c();
      CHECK(st == FH_OK || st == FH_ERR_INVALID_ARG || st == FH_ERR_UNSUPPORTED);
      if (t == 9) CHECK(st != FH_OK);
      if (x < 0) CHECK(st == FH_ERR_INVALID_ARG || t == 9);
    }
}
template <typename C>
static void ends32(int32_t C::*arg) {
  for (int32_t x : kEnds32) {
    C c;
    c.*arg = x;
    const int st = c();
    CHECK(st == FH_OK || st == FH_ERR_INVALID_ARG || st == FH_ERR_UNSUPPORTED);
  }
}
// strides whose rows would lie past any address, and whose bytes come back to a
// multiple of 16 in 64 bits
template <typename C>
static void no_memory(int64_t C::*ld) {
  for (int t : {FH_DTYPE_BF16, FH_DTYPE_F32})
    for (int s : {60, 61, 62}) {
      C c;
      c.dtype = t;
      c.*ld = ((int64_t)1 << s) + 256;
      if ((((int64_t)1 << s) + 256) < 0) continue;
      CHECK(c() == FH_ERR_UNSUPPORTED);
    }
}

int main() {
  CHECK(Norm()() == FH_OK && Quantize()() == FH_OK && Logits()() == FH_OK && Verify()() == FH_OK);
  for (auto p : {&Norm::ldx, &Norm::ldr, &Norm::ldro, &Norm::ldy, &Norm::ldy8, &Norm::lds}) {
    ends64(p);
    // 4 rows apart by 2^60 fp32 values and more: past the address space
    for (int s : {61, 62}) {
      Norm c;
      c.dtype = FH_DTYPE_F32;
      c.*p = ((int64_t)1 << s) + 256;
      CHECK(c() == FH_ERR_UNSUPPORTED);
      // one row: a stride is not looked at
      c.rows = 1;
      CHECK(c() == FH_OK);
    }
  }
  ends64(&Norm::rows);
  ends32(&Norm::d);
  for (auto p : {&Quantize::lde, &Quantize::lde8, &Quantize::lds}) {
    ends64(p);
    no_memory(p);
  }
  ends64(&Quantize::v);
  ends32(&Quantize::d);
  for (auto p : {&Logits::ldh, &Logits::lds, &Logits::lde, &Logits::ldes, &Logits::ldo}) {
    ends64(p);
    no_memory(p);
  }
  ends64(&Logits::v);
  ends32(&Logits::d);
  ends32(&Logits::rows);
  for (auto p : {&Verify::ldl, &Verify::ldq}) {
    ends64(p);
    no_memory(p);
  }
  ends64(&Verify::rows);
  ends64(&Verify::v);
  ends64(&Verify::n);
  ends32(&Verify::B);
  ends32(&Verify::m);
  ends32(&Verify::mode);
  for (float x : {0.0f, -0.0f, -1.0f, NAN, INFINITY, -INFINITY}) {
    Verify c;
    c.tau = x;
    CHECK(c() == FH_ERR_INVALID_ARG);
  }
  for (float x : {-1.0f, NAN, INFINITY, -INFINITY}) {
    Norm c;
    c.eps = x;
    CHECK(c() == FH_ERR_INVALID_ARG);
  }
  printf("ok %d\n", g_checks);
  return 0;
}
