// Verification of drafted tokens against the target's logits from given
// uniform numbers.  For the drafts x_1 .. x_n of a sequence, with
// p_i = softmax(z_i / tau) at the sequence's i-th row and q_i the draft's
// probabilities (one-hot at x_i when none are given):
//   x_i is accepted while u_i q_i(x_i) < p_i(x_i);
//   the token after the accepted ones is drawn from max(p - q, 0) at the row
//   of the first rejection, or from p at row n + 1 when all are accepted;
//   a draw is the smallest t with C_t > u C_v, C the running sum of the weights.
// Greedy: x_i is accepted while it is its row's argmax, which is also the
// token after the accepted ones.
//
// The weights, their sums and the tests are in fp64: neighbouring C_t lie
// about 1 / v of the total apart, 8e-6 at v = 128256, so a running sum in fp32
// (errors of 1e-6) would draw another token than the given u says in a few of
// a hundred calls.
//
// First launch, per (row, chunk): the maximum, its index and the sum of
// exponentials.  Second, per sequence: the decisions, folded from the chunks'
// records, then the draw, for which the chunks' sums name the chunk and that
// chunk's running sum the token.  Only max(p - q, 0) has other chunk sums than
// p: then a workgroup per chunk sums the chunk's weights, and the sequence's
// last one draws.  Those decide for themselves in the second launch where
// they all fit the device at once (one sequence of four drafts, 128256: 5 + 9
// us); where they do not, a third launch takes over the second's state (64
// sequences: 31 + 8 + 18 us; with the same decisions made by every chunk's
// workgroup the second launch took 41).  Greedy decoding of as many rows: 31 + 5.
#include "fh_device.h"
#include "fh_internal.h"

namespace fh {

namespace {

constexpr int kVThreads = 256;  // of the first launch
constexpr int kVWaves = kVThreads / kWave;
// A chunk is 8 values a thread of the draws; the decisions have a wave for each
// of 8 rows.
constexpr int kDrawThreads = kVerifyChunk / 8, kDecideThreads = 512;

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

// a.empty[s] = the sequences before s that have no row and so take none of the
// places that rows without a draft have (one workgroup, a quarter of the
// sequences a wave); 0 where the arrays are too short for the drafts of all
// sequences one after the other.
__device__ __forceinline__ void count_empty(const VerifyArgs& a, int w, int lane) {
  __shared__ int s_count[kVWaves];
  const int64_t per = ((a.B + kVWaves - 1) / kVWaves + kWave - 1) / kWave * kWave;
  const int64_t from = w * per < a.B ? w * per : a.B;
  const int64_t to = from + per < a.B ? from + per : a.B;
  auto none = [&](int64_t s) { return s < to && a.row_start[s + 1] <= a.row_start[s]; };
  int count = 0;
#pragma unroll 4
  for (int64_t s = from; s < to; s += kWave)
    count += __builtin_popcountll(__ballot(none(s + lane)));
  if (lane == 0) s_count[w] = count;
  __syncthreads();
  int before = 0, total = 0;
  for (int i = 0; i < kVWaves; ++i) {
    before += i < w ? s_count[i] : 0;
    total += s_count[i];
  }
  const bool whole = a.n_drafts >= (int64_t)a.row_start[a.B] - (a.B - total);
  for (int64_t s = from; s < to; s += kWave) {
    const uint64_t m = __ballot(none(s + lane));
    if (s + lane < to)
      a.empty[s + lane] =
          whole ? before + __builtin_popcountll(m & ((1ull << lane) - 1)) : 0;
    before += __builtin_popcountll(m);
  }
}

// The record of a (row, chunk), one wave each: top = the maximum, best = its
// lowest index (kBest; greedy decoding), sum = the sum of exp((z - top) / tau).
// A NaN or +inf logit makes the sum NaN; a chunk of -inf alone has sum 0.
// A lane holds 32 values, so that the wave's reductions are a tenth of the
// work, and no wave waits for another.  The first workgroup counts the empty
// sequences instead.
template <typename T, bool kBest>
__global__ __launch_bounds__(kVThreads) void verify_rows_kernel(const VerifyArgs a) {
  constexpr int U = kVerifyChunk / (kWave * 8);
  const int tid = threadIdx.x, lane = tid & 63;
  // the next launch counts the workgroups of a sequence from zero
  for (int64_t s = (int64_t)blockIdx.x * kVThreads + tid; s < a.B;
       s += (int64_t)gridDim.x * kVThreads)
    a.arrived[s] = 0u;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  if (blockIdx.x == 0) {
    count_empty(a, w, lane);
    return;
  }
  const int64_t id = (int64_t)(blockIdx.x - 1) * kVWaves + w;
  const int64_t r = id / a.nchunk;
  if (r >= a.rows) return;
  const uint8_t* row = a.logits + r * a.l_bytes;
  const int64_t c0 = (id - r * a.nchunk) * kVerifyChunk;
  const int64_t end = c0 + kVerifyChunk < a.v ? c0 + kVerifyChunk : a.v;
  float x[U][8];
  float top = -INFINITY;
  bool nan = false;
  if (c0 + kVerifyChunk <= a.v) {
#pragma unroll
    for (int i = 0; i < U; ++i) load_whole8<T>(row, c0 + (i * kWave + lane) * 8, x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i)
      load8<T>(row, c0 + (i * kWave + lane) * 8, end, -INFINITY, x[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      top = fmaxf(top, fmaxf(x[i][j], x[i][j + 1]));
      nan |= __builtin_isunordered(x[i][j], x[i][j + 1]);
    }
  top = wave_max(nan ? INFINITY : top);  // (a NaN ends as +inf does)
  double sum = 0.0;
  int best = INT32_MAX;
  if (top == INFINITY) {
    sum = NAN;
  } else if (top > -INFINITY) {
    double part[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[j & 1] += weight<false>(x[i][j], top, a.k, a.lo);
    sum = wave_sum_f64(part[0] + part[1]);
    if constexpr (kBest) {
#pragma unroll
      for (int i = U - 1; i >= 0; --i)
#pragma unroll
        for (int j = 7; j >= 0; --j)
          if (x[i][j] == top) best = (int)(c0 + (i * kWave + lane) * 8 + j);
      best = (int)~wave_max_u32(~(uint32_t)best);
    }
  }
  if (lane == 0) a.part[id] = VerifyPart{sum, top, best};
}

// A row's maximum, lowest argmax and sum from its chunks' records (one wave).
struct RowFold {
  float top;
  int best;
  double sum;
};
// a chunk's sum, relative to the row's maximum (a chunk without a value has
// sum 0)
__device__ __forceinline__ double chunk_sum(const VerifyPart& p, float top, double k) {
  return p.top == -INFINITY ? 0.0 : p.sum * weight(p.top, top, k);
}
__device__ __forceinline__ RowFold fold_row(const VerifyArgs& a, int64_t r, int lane) {
  const VerifyPart* part = a.part + r * a.nchunk;
  RowFold f{-INFINITY, INT32_MAX, 0.0};
  if (a.nchunk <= kWave) {
    const VerifyPart p =
        lane < a.nchunk ? part[lane] : VerifyPart{0.0, -INFINITY, INT32_MAX};
    f.top = wave_max(p.top);
    f.sum = chunk_sum(p, f.top, a.k);
    f.best = p.top == f.top ? p.best : INT32_MAX;
  } else {
    for (int c = lane; c < a.nchunk; c += kWave) f.top = fmaxf(f.top, part[c].top);
    f.top = wave_max(f.top);
    for (int c = lane; c < a.nchunk; c += kWave) {
      const VerifyPart p = part[c];
      f.sum += chunk_sum(p, f.top, a.k);
      if (p.top == f.top && p.best < f.best) f.best = p.best;
    }
  }
  f.sum = wave_sum_f64(f.sum);
  f.best = (int)~wave_max_u32(~(uint32_t)f.best);
  return f;
}

__device__ __forceinline__ float log_prob(float x, const RowFold& f, double k) {
  return (float)(((double)x - (double)f.top) * (k * 0.693147180559945309) - log(f.sum));
}

// The weights of 8 values (p, or what q leaves of it, or p without a token)
// from t on, and their sum; x: the logits.
template <typename T>
struct Weights {
  const uint8_t* row;
  const uint8_t* q;   // null: none
  int64_t skip;       // -1: none
  float top;
  double k, scale;    // scale 1 / sum where q is subtracted, else 1
  __device__ __forceinline__ double at(int64_t t, int64_t end, float* x, double* w) const {
    float y[8];
    load8<T>(row, t, end, -INFINITY, x);
    if (q) load8<float>(q, t, end, 0.0f, y);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double p = weight(x[j], top, k) * scale;
      if (q)
        p = fmax(p - (double)y[j], 0.0);
      else if (t + j == skip)
        p = 0.0;
      w[j] = p;
      sum += p;
    }
    return sum;
  }
};

enum VerifyMode { kAll, kDecide, kDraw };

// kAll: a workgroup per (sequence, chunk); kDecide: one per sequence, which
// also draws unless q is to be subtracted; kDraw: per (sequence, chunk), the
// draws that kDecide left.
constexpr int decide_threads(VerifyMode m) { return m == kDraw ? kDrawThreads : kDecideThreads; }
template <typename T, VerifyMode kMode>
__global__ __launch_bounds__(decide_threads(kMode)) void verify_decide_kernel(const VerifyArgs a) {
  constexpr int kDThreads = decide_threads(kMode), kDWaves = kDThreads / kWave;
  __shared__ int s_last[kDWaves];   // 0: the wave's draft was accepted
  __shared__ RowFold s_fold[kDWaves];
  __shared__ int s_token[kDWaves];
  __shared__ float s_logp[kDWaves];
  __shared__ double s_sum[kDWaves];
  __shared__ int s_pass[kDWaves];
  __shared__ int s_go, s_chunk, s_plain;
  __shared__ double s_need;
  const int tid = threadIdx.x, lane = tid & 63, w = tid / kWave;
  const int per = kMode == kDecide ? 1 : a.nchunk;  // workgroups a sequence
  const int s = blockIdx.x / (unsigned)per, chunk = blockIdx.x % (unsigned)per;
  int32_t* out = a.out_tokens + (int64_t)s * a.max_tokens;
  float* logp = a.out_logp ? a.out_logp + (int64_t)s * a.max_tokens : nullptr;
  int64_t row, draft;   // what is drawn from
  int at;               // accepted drafts
  bool rejected;
  RowFold f;
  if constexpr (kMode == kDraw) {
    const VerifyState st = a.state[s];
    if (!st.draws) return;
    row = st.row;
    draft = st.draft;
    at = st.at;
    rejected = true;
    f = RowFold{st.top, 0, st.sum};
  } else {
    const bool writer = chunk == 0;
    const int64_t r0 = a.row_start[s], r1 = a.row_start[s + 1];
    const int64_t d0 = r0 - s + a.empty[s];  // the sequence's first draft
    const int64_t n = r1 - r0 - 1;     // its drafts
    bool bad = r0 < 0 || n < 0 || r1 > a.rows || n >= a.max_tokens || d0 < 0 ||
               d0 + n > a.n_drafts;
    int64_t base = 0;
    if (!bad) {
      bool far = false;
      for (int64_t i = tid; i < n; i += kDThreads) {
        const int x = a.draft_tokens[d0 + i];
        far |= x < 0 || (int64_t)x >= a.v;
      }
      // the rows in order, eight at a time, up to the first whose draft is not
      // taken
      for (;; base += kDWaves) {
        const int64_t i = base + w;
        if (i <= n) {
          // (requested together with the records; a draft outside the
          // vocabulary is seen to below)
          const int x = i < n ? a.draft_tokens[d0 + i] : 0;
          const int64_t xi = x < 0 ? 0 : (int64_t)x < a.v ? x : a.v - 1;
          const float z = load1<T>(a.logits + (r0 + i) * a.l_bytes, xi);
          const float q = a.q && i < n ? a.q[(d0 + i) * a.ldq + xi] : 1.0f;
          const float u = a.sample && i < n ? a.u_accept[d0 + i] : 0.0f;
          const RowFold g = fold_row(a, r0 + i, lane);
          if (lane == 0) {
            bool take = i < n && g.sum > 0.0 && g.sum < INFINITY;
            if (take)
              take = a.sample ? (double)u * (double)q * g.sum < weight(z, g.top, a.k)
                              : x == g.best;
            s_last[w] = !take;
            s_fold[w] = g;
            s_token[w] = x;
            if (logp && take && writer) s_logp[w] = log_prob(z, g, a.k);
          }
        }
        if (base == 0)
          bad = __syncthreads_or(far);
        else
          __syncthreads();
        if (bad) break;
        int hit = -1;
        for (int k = 0; k < kDWaves && base + k <= n; ++k)
          if (hit < 0 && s_last[k]) hit = k;
        if (writer && tid < (hit >= 0 ? hit : kDWaves)) {
          out[base + tid] = s_token[tid];
          if (logp) logp[base + tid] = s_logp[tid];
        }
        if (hit >= 0) {
          at = (int)base + hit;
          f = s_fold[hit];
          break;
        }
        __syncthreads();
      }
    }
    if (bad) {
      if (writer) {
        for (int i = tid; i < a.max_tokens; i += kDThreads) {
          out[i] = -1;
          if (logp) logp[i] = 0.0f;
        }
        if (tid == 0) {
          a.out_accepted[s] = -1;
          if (kMode == kDecide && a.q) a.state[s].draws = 0;
        }
      }
      return;
    }
    const bool some = f.sum > 0.0 && f.sum < INFINITY;  // the row has a distribution
    rejected = at < n;
    row = r0 + at;
    draft = d0 + at;
    if (writer) {
      for (int64_t i = at + 1 + tid; i < a.max_tokens; i += kDThreads) {
        out[i] = -1;
        if (logp) logp[i] = 0.0f;
      }
      if (tid == 0) {
        a.out_accepted[s] = at;
        if (!some || !a.sample) {
          out[at] = some ? f.best : -1;
          if (logp) logp[at] = some ? log_prob(f.top, f, a.k) : 0.0f;
        }
        if (kMode == kDecide && a.q)
          a.state[s] = VerifyState{row, draft, f.sum, f.top, at, some && rejected};
      }
    }
    if (!some || !a.sample) return;
    if (rejected && a.q ? kMode == kDecide : !writer) return;
  }

  Weights<T> wt;
  wt.row = a.logits + row * a.l_bytes;
  wt.q = rejected && a.q ? reinterpret_cast<const uint8_t*>(a.q + draft * a.ldq) : nullptr;
  wt.skip = rejected && !a.q ? a.draft_tokens[draft] : -1;
  wt.top = f.top;
  wt.k = a.k;
  wt.scale = wt.q ? 1.0 / f.sum : 1.0;
  double* pw = a.part_weight + (int64_t)s * a.nchunk;
  float x[8];
  double y[8];
  // this thread's first value of a chunk, and the chunk's end (threads behind
  // the chunk have nothing of it)
  auto end_of = [&](int c) {
    const int64_t e = (int64_t)(c + 1) * kVerifyChunk;
    return e < a.v ? e : a.v;
  };
  auto first_of = [&](int c) {
    return tid < kDrawThreads ? (int64_t)c * kVerifyChunk + tid * 8 : end_of(c);
  };
  // a chunk's weights, this thread's 8 of them in y; the sum is thread 0's
  auto chunk_weight = [&](int c) {
    double sum = wave_sum_f64(wt.at(first_of(c), end_of(c), x, y));
    if (lane == 0) s_sum[w] = sum;
    __syncthreads();
    if (tid == 0)
      for (int i = 1; i < kDWaves; ++i) sum += s_sum[i];
    return sum;
  };
  if (wt.q) {
    const double sum = chunk_weight(chunk);
    if (tid == 0) {
      // Seen by the whole device before the count goes up; whoever counts the
      // last one finds all of them.
      __hip_atomic_store(reinterpret_cast<uint64_t*>(pw + chunk),
                         (uint64_t)__double_as_longlong(sum), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint32_t before = __hip_atomic_fetch_add(a.arrived + s, 1u, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT);
      s_go = before + 1 == (uint32_t)per;
    }
    __syncthreads();
    if (!s_go) return;
  }
  // a token that p loses: its chunk's sum without it
  const int skip_chunk = wt.skip >= 0 ? (int)(wt.skip / kVerifyChunk) : -1;
  double skip_sum = 0.0;
  if (skip_chunk >= 0) skip_sum = chunk_weight(skip_chunk);

  // the chunk: the first whose running sum passes u times the total
  if (w == 0) {
    skip_sum = lane_f64(skip_sum, 0);
    const VerifyPart* part = a.part + row * a.nchunk;
    auto get = [&](int c, bool plain) {
      if (c >= a.nchunk) return 0.0;
      if (!plain && wt.q)
        return __longlong_as_double((long long)__hip_atomic_load(
            reinterpret_cast<uint64_t*>(pw + c), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      if (!plain && c == skip_chunk) return skip_sum;
      return chunk_sum(part[c], f.top, a.k);
    };
    const float u = a.u_sample[s];
    bool plain = !rejected;
    double total = 0.0;
    for (;;) {
      total = 0.0;
      for (int c = lane; c < a.nchunk; c += kWave) total += get(c, plain);
      total = wave_sum_f64(total);
      if (plain || total > 0.0) break;
      plain = true;  // nothing is left of p: the draw is from p itself
    }
    const double target = fmax((double)u, 0.0) * total;
    double before = 0.0, need = 0.0;
    int end = 0;   // the chunk, or the last one with a weight
    bool hit = false;
    for (int c0 = 0; c0 < a.nchunk && !hit; c0 += kWave) {
      const double p = get(c0 + lane, plain);
      const double scan = before + wave_scan_f64(p);
      const uint64_t over = __ballot(p > 0.0 && scan > target), some = __ballot(p > 0.0);
      // (rounding can leave no chunk over the target: then the last one, with
      // a need that its running sum may not pass either)
      const int l = over ? (int)__builtin_ctzll(over) : some ? 63 - __builtin_clzll(some) : -1;
      if (l >= 0) {
        end = c0 + l;
        need = target - lane_f64(scan - p, l);
        hit = over != 0;
      }
      before = lane_f64(scan, 63);
    }
    if (lane == 0) {
      s_chunk = end;
      s_plain = plain;
      s_need = need;
    }
  }
  __syncthreads();
  if (s_plain) {
    wt.q = nullptr;
    wt.skip = -1;
    wt.scale = 1.0;
  }
  // the token: the first whose running sum passes what is left of the target
  const double need = s_need;
  const int64_t t = first_of(s_chunk);
  const double sum = wt.at(t, end_of(s_chunk), x, y);
  const double scan = wave_scan_f64(sum);
  if (lane == 63) s_sum[w] = scan;
  __syncthreads();
  double c = scan - sum;
  for (int k = 0; k < w; ++k) c += s_sum[k];
  int hit = -1, last = -1;
  float hit_x = 0.0f, last_x = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c += y[j];
    if (y[j] > 0.0) {
      last = (int)(t + j);
      last_x = x[j];
      if (c > need && hit < 0) {
        hit = last;
        hit_x = x[j];
      }
    }
  }
  // tokens rise with the lane and the wave: the first wave's first lane that
  // passed, or (where rounding left none) the last one's last with a weight
  const uint64_t hits = __ballot(hit >= 0), lasts = __ballot(last >= 0);
  if (lane == 0) s_pass[w] = (hits ? 1 : 0) | (lasts ? 2 : 0);
  __syncthreads();
  int first = -1, end = -1;
  for (int k = kDWaves - 1; k >= 0; --k) {
    if (s_pass[k] & 1) first = k;
    if ((s_pass[k] & 2) && end < 0) end = k;
  }
  const bool mine = first >= 0 ? w == first && lane == (int)__builtin_ctzll(hits | 1ull << 63)
                               : w == end && lane == 63 - (int)__builtin_clzll(lasts | 1ull);
  if (mine) {
    out[at] = first >= 0 ? hit : last;
    if (logp) logp[at] = log_prob(first >= 0 ? hit_x : last_x, f, a.k);
  }
}

template <typename T>
void enqueue(const VerifyArgs& a, hipStream_t s) {
  const unsigned n = (unsigned)a.nchunk, B = (unsigned)a.B;
  const dim3 rows((unsigned)((a.rows * a.nchunk + kVWaves - 1) / kVWaves) + 1);
  if (a.rows && a.sample)
    hipLaunchKernelGGL((verify_rows_kernel<T, false>), rows, dim3(kVThreads), 0, s, a);
  else if (a.rows)
    hipLaunchKernelGGL((verify_rows_kernel<T, true>), rows, dim3(kVThreads), 0, s, a);
  // Two workgroups a compute unit fit the device at once.  Calls with two and
  // with three launches, us: 8 sequences of 128256 (504 workgroups) 18.0 and 21.3,
  // 16 (1008) 22.7 and 24.9, 32 (2016) 31.7 and 29.0; 32 of 32000 (512) 17.2 and
  // 20.9, 40 (640) 22.1 and 21.5, 128 (2048) 49 and 29.
  if (a.q && (int64_t)B * n <= 512) {
    hipLaunchKernelGGL((verify_decide_kernel<T, kAll>), dim3(B * n), dim3(kDecideThreads), 0, s, a);
    return;
  }
  hipLaunchKernelGGL((verify_decide_kernel<T, kDecide>), dim3(B), dim3(kDecideThreads), 0, s, a);
  if (a.q)
    hipLaunchKernelGGL((verify_decide_kernel<T, kDraw>), dim3(B * n), dim3(kDrawThreads), 0, s, a);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s) {
  if (dtype == FH_DTYPE_BF16)
    enqueue<uint16_t>(a, s);
  else
    enqueue<float>(a, s);
  return hipGetLastError();
}

}  // namespace fh
