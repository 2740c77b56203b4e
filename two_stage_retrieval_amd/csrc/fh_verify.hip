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
// Three launches: per (row, chunk) the maximum, its index and the sum of
// exponentials; per (sequence, chunk) the decisions, folded from the chunks'
// records by every workgroup for itself, and the sum of the chosen row's
// weights; per sequence the chunk that holds the draw and the token in it.
#include "fh_device.h"
#include "fh_internal.h"

namespace fh {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWaves = kVThreads / kWave;

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, kWave);
  return x;
}

// exp(x / tau) for x <= 0, k = 1 / tau
__device__ __forceinline__ double weight(float x, float top, double k) {
  return exp(((double)x - (double)top) * k);
}

// Values [i, i + 8) of a row of n; past its end -inf (logits) or 0
// (probabilities), without reading there.
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* row, int64_t i, int64_t n, float fill,
                                      float* x) {
  if (i + 8 <= n) {
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

// Per (row, chunk): top = the maximum, best = its lowest index, sum = the sum
// of exp((z - top) / tau).  A NaN or +inf logit makes the sum NaN; a chunk of
// -inf alone has sum 0.
template <typename T>
__global__ __launch_bounds__(kVThreads) void verify_rows_kernel(const VerifyArgs a) {
  __shared__ float s_top[kVWaves];
  __shared__ double s_sum[kVWaves];
  __shared__ int s_best[kVWaves];
  const int tid = threadIdx.x, w = tid / kWave;
  const int64_t r = blockIdx.x / (unsigned)a.nchunk;
  const int chunk = blockIdx.x % (unsigned)a.nchunk;
  const uint8_t* row = a.logits + r * a.l_bytes;
  const int64_t c0 = (int64_t)chunk * a.chunk;
  const int64_t end = c0 + a.chunk < a.v ? c0 + a.chunk : a.v;
  float x[kVerifyMaxUnits][8];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVerifyMaxUnits; ++i) {
    load8<T>(row, c0 + (i * kVThreads + tid) * 8, i < a.units ? end : 0, -INFINITY, x[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[i][j]);
  }
  top = wave_max(top);
  if ((tid & 63) == 0) s_top[w] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kVWaves; ++i) top = fmaxf(top, s_top[i]);
  double sum = 0.0;
  int best = INT32_MAX;
  if (top == -INFINITY) {  // all masked, or NaN: exp would make NaN of both
#pragma unroll
    for (int i = 0; i < kVerifyMaxUnits; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x[i][j] != x[i][j]) sum = NAN;
  } else {
#pragma unroll
    for (int i = 0; i < kVerifyMaxUnits; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum += weight(x[i][j], top, a.inv_tau);
        if (x[i][j] == top) {
          const int t = (int)(c0 + (i * kVThreads + tid) * 8 + j);
          best = t < best ? t : best;
        }
      }
    }
  }
  sum = wave_sum_f64(sum);
  best = (int)~wave_max_u32(~(uint32_t)best);
  if ((tid & 63) == 0) {
    s_sum[w] = sum;
    s_best[w] = best;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kVWaves; ++i) {
      sum += s_sum[i];
      best = s_best[i] < best ? s_best[i] : best;
    }
    const int64_t o = r * a.nchunk + chunk;
    a.part_top[o] = top;
    a.part_sum[o] = sum;
    a.part_best[o] = best;
  }
}

// A row's maximum, lowest argmax and sum from its chunks' records (one wave).
struct RowFold {
  float top;
  int best;
  double sum;
};
__device__ __forceinline__ RowFold fold_row(const VerifyArgs& a, int64_t r, int lane) {
  const int64_t o = r * a.nchunk;
  RowFold f{-INFINITY, INT32_MAX, 0.0};
  for (int c = lane; c < a.nchunk; c += kWave) f.top = fmaxf(f.top, a.part_top[o + c]);
  f.top = wave_max(f.top);
  for (int c = lane; c < a.nchunk; c += kWave) {
    const float t = a.part_top[o + c];
    const double s = a.part_sum[o + c];
    // a chunk without a value (sum 0) adds nothing; its NaN stays
    f.sum += t == -INFINITY ? s : s * weight(t, f.top, a.inv_tau);
    if (t == f.top && a.part_best[o + c] < f.best) f.best = a.part_best[o + c];
  }
  f.sum = wave_sum_f64(f.sum);
  f.best = (int)~wave_max_u32(~(uint32_t)f.best);
  return f;
}

__device__ __forceinline__ float log_prob(float x, const RowFold& f, double k) {
  return (float)(((double)x - (double)f.top) * k - log(f.sum));
}

// Per (sequence, chunk): the decisions and, for a sample, the sum of the
// chosen row's weights over the chunk.
template <typename T>
__global__ __launch_bounds__(kVThreads) void verify_decide_kernel(const VerifyArgs a) {
  __shared__ int s_state[kVWaves];   // 0 accepted, 1 the sequence's last token is drawn here
  __shared__ RowFold s_fold[kVWaves];
  __shared__ int s_token[kVWaves];
  __shared__ float s_logp[kVWaves];
  __shared__ double s_sum[kVWaves];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 63, w = tid / kWave;
  const int per = a.sample ? a.nchunk : 1;  // workgroups a sequence
  const int s = blockIdx.x / (unsigned)per, chunk = blockIdx.x % (unsigned)per;
  const int64_t r0 = a.row_start[s], r1 = a.row_start[s + 1];
  const int64_t d0 = r0 - s;         // the sequence's first draft
  const int64_t n = r1 - r0 - 1;     // its drafts
  bool bad = r0 < 0 || n < 0 || r1 > a.rows || n >= a.max_tokens || d0 < 0 ||
             d0 + n > a.n_drafts;
  if (!bad) {
    if (tid == 0) s_bad = 0;
    __syncthreads();
    for (int64_t i = tid; i < n; i += kVThreads) {
      const int x = a.draft_tokens[d0 + i];
      if (x < 0 || (int64_t)x >= a.v) s_bad = 1;
    }
    __syncthreads();
    bad = s_bad != 0;
  }
  const bool writer = chunk == 0;
  int32_t* out = a.out_tokens + (int64_t)s * a.max_tokens;
  float* logp = a.out_logp ? a.out_logp + (int64_t)s * a.max_tokens : nullptr;
  VerifyState* st = a.state + s;
  if (bad) {
    if (writer) {
      for (int i = tid; i < a.max_tokens; i += kVThreads) {
        out[i] = -1;
        if (logp) logp[i] = 0.0f;
      }
      if (tid == 0) {
        a.out_accepted[s] = -1;
        st->kind = kVerifyDone;
      }
    }
    return;
  }
  int64_t at = 0;
  RowFold f;
  for (int64_t base = 0;; base += kVWaves) {
    const int64_t i = base + w;
    if (i <= n) {
      const RowFold g = fold_row(a, r0 + i, lane);
      if (lane == 0) {
        int last = 1;
        if (i < n) {
          const int x = a.draft_tokens[d0 + i];
          const float z = load1<T>(a.logits + (r0 + i) * a.l_bytes, x);
          bool take = false;
          if (g.sum > 0.0 && g.sum < INFINITY) {
            if (a.sample) {
              const double q = a.q ? (double)a.q[(d0 + i) * a.ldq + x] : 1.0;
              take = (double)a.u_accept[d0 + i] * q < weight(z, g.top, a.inv_tau) / g.sum;
            } else {
              take = x == g.best;
            }
          }
          if (take) {
            last = 0;
            s_token[w] = x;
            if (logp) s_logp[w] = log_prob(z, g, a.inv_tau);
          }
        }
        s_state[w] = last;
        s_fold[w] = g;
      }
    }
    __syncthreads();
    int hit = -1;
    for (int k = 0; k < kVWaves && base + k <= n; ++k)
      if (hit < 0 && s_state[k]) hit = k;
    if (writer && tid < (hit >= 0 ? hit : kVWaves)) {
      out[base + tid] = s_token[tid];
      if (logp) logp[base + tid] = s_logp[tid];
    }
    if (hit >= 0) {
      at = base + hit;
      f = s_fold[hit];
      break;
    }
    __syncthreads();
  }
  const bool valid = f.sum > 0.0 && f.sum < INFINITY;
  const bool rejected = at < n;
  if (writer) {
    // a sample's token is the next launch's
    const int final_token = valid && !a.sample ? f.best : -1;
    for (int64_t i = at + tid; i < a.max_tokens; i += kVThreads) {
      out[i] = i == at ? final_token : -1;
      if (logp) logp[i] = i == at && final_token >= 0 ? log_prob(f.top, f, a.inv_tau) : 0.0f;
    }
    if (tid == 0) {
      a.out_accepted[s] = (int)at;
      st->kind = valid && a.sample ? (rejected ? kVerifyResidual : kVerifyPlain) : kVerifyDone;
      st->at = (int)at;
      st->row = r0 + at;
      st->draft = d0 + at;
      st->top = f.top;
      st->sum = f.sum;
    }
  }
  if (!a.sample || !valid || !rejected) return;
  // the chunk's part of the residual weights
  const uint8_t* row = a.logits + (r0 + at) * a.l_bytes;
  const uint8_t* q = a.q ? reinterpret_cast<const uint8_t*>(a.q + (d0 + at) * a.ldq) : nullptr;
  const int64_t skip = a.q ? -1 : a.draft_tokens[d0 + at];
  const int64_t c0 = (int64_t)chunk * a.chunk;
  const int64_t end = c0 + a.chunk < a.v ? c0 + a.chunk : a.v;
  double sum = 0.0;
  for (int i = 0; i < a.units; ++i) {
    const int64_t t = c0 + (i * kVThreads + tid) * 8;
    float x[8], y[8];
    load8<T>(row, t, end, -INFINITY, x);
    if (q) load8<float>(q, t, end, 0.0f, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double p = weight(x[j], f.top, a.inv_tau) / f.sum;
      sum += q ? fmax(p - (double)y[j], 0.0) : (t + j == skip ? 0.0 : p);
    }
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) s_sum[w] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kVWaves; ++i) sum += s_sum[i];
    a.part_weight[(int64_t)s * a.nchunk + chunk] = sum;
  }
}

// Per sequence that draws: the chunk and the token.
template <typename T>
__global__ __launch_bounds__(kVThreads) void verify_draw_kernel(const VerifyArgs a) {
  __shared__ double s_sum[kVWaves];
  __shared__ double s_before;
  __shared__ int s_chunk, s_plain, s_token, s_last;
  const int tid = threadIdx.x, lane = tid & 63, w = tid / kWave;
  const int s = blockIdx.x;
  const VerifyState st = a.state[s];
  if (st.kind == kVerifyDone) return;
  const double* pw = a.part_weight + (int64_t)s * a.nchunk;
  const int64_t o = st.row * a.nchunk;
  // a chunk's share under p
  auto share = [&](int c) {
    const float t = a.part_top[o + c];
    return t == -INFINITY ? 0.0 : a.part_sum[o + c] * weight(t, st.top, a.inv_tau) / st.sum;
  };
  if (tid == 0) {
    bool plain = st.kind == kVerifyPlain;
    double total = 0.0;
    if (!plain) {
      for (int c = 0; c < a.nchunk; ++c) total += pw[c];
      plain = !(total > 0.0);  // q covers p everywhere: draw from p
    }
    if (plain) {
      total = 0.0;
      for (int c = 0; c < a.nchunk; ++c) total += share(c);
    }
    const double target = fmax((double)a.u_sample[s], 0.0) * total;
    double before = 0.0;
    int hit = -1, last = 0;
    double last_before = 0.0;
    for (int c = 0; c < a.nchunk && hit < 0; ++c) {
      const double x = plain ? share(c) : pw[c];
      if (before + x > target) hit = c;
      if (x > 0.0) { last = c; last_before = before; }
      if (hit < 0) before += x;
    }
    if (hit < 0) { hit = last; before = last_before; }
    s_chunk = hit;
    s_plain = plain;
    s_before = target - before;  // what the chunk's running sum has to pass
    s_token = INT32_MAX;
    s_last = -1;
  }
  __syncthreads();
  const bool plain = s_plain;
  const double need = s_before;
  const uint8_t* row = a.logits + st.row * a.l_bytes;
  const uint8_t* q =
      a.q && !plain ? reinterpret_cast<const uint8_t*>(a.q + st.draft * a.ldq) : nullptr;
  const int64_t skip = a.q || plain ? -1 : a.draft_tokens[st.draft];
  const int64_t c0 = (int64_t)s_chunk * a.chunk;
  const int64_t end = c0 + a.chunk < a.v ? c0 + a.chunk : a.v;
  double before = 0.0;
  for (int i = 0; i < a.units; ++i) {
    const int64_t t = c0 + (i * kVThreads + tid) * 8;
    float x[8], y[8];
    double wt[8], sum = 0.0;
    load8<T>(row, t, end, -INFINITY, x);
    if (q) load8<float>(q, t, end, 0.0f, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double p = weight(x[j], st.top, a.inv_tau) / st.sum;
      wt[j] = q ? fmax(p - (double)y[j], 0.0) : (t + j == skip ? 0.0 : p);
      sum += wt[j];
    }
    // running sum before this thread's values
    double scan = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double up = __shfl_up(scan, d, kWave);
      if (lane >= d) scan += up;
    }
    if (lane == 63) s_sum[w] = scan;
    __syncthreads();
    double c = before + (scan - sum);
    for (int k = 0; k < w; ++k) c += s_sum[k];
    for (int k = 0; k < kVWaves; ++k) before += s_sum[k];
    int hit = INT32_MAX, last = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c += wt[j];
      if (wt[j] > 0.0) {
        last = (int)(t + j);
        if (c > need && hit == INT32_MAX) hit = (int)(t + j);
      }
    }
    if (hit != INT32_MAX) atomicMin(&s_token, hit);
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    if (s_token != INT32_MAX) break;
  }
  if (tid == 0) {
    const int t = s_token != INT32_MAX ? s_token : s_last;
    const int64_t i = (int64_t)s * a.max_tokens + st.at;
    a.out_tokens[i] = t;
    if (a.out_logp && t >= 0) {
      const RowFold f{st.top, 0, st.sum};
      a.out_logp[i] = log_prob(load1<T>(row, t), f, a.inv_tau);
    }
  }
}

template <typename T>
void enqueue(const VerifyArgs& a, int B, hipStream_t s) {
  const dim3 block(kVThreads);
  const unsigned n = (unsigned)a.nchunk;
  if (a.rows)
    hipLaunchKernelGGL(verify_rows_kernel<T>, dim3((unsigned)a.rows * n), block, 0, s, a);
  hipLaunchKernelGGL(verify_decide_kernel<T>, dim3((unsigned)B * (a.sample ? n : 1u)), block, 0, s,
                     a);
  if (a.sample) hipLaunchKernelGGL(verify_draw_kernel<T>, dim3((unsigned)B), block, 0, s, a);
}

}  // namespace

void plan_verify(VerifyArgs& a) {
  a.units = 2;
  a.chunk = (int64_t)a.units * kVThreads * 8;
  a.nchunk = (int)((a.v + a.chunk - 1) / a.chunk);
}

hipError_t launch_verify(const VerifyArgs& a, int dtype, int B, hipStream_t s) {
  if (dtype == FH_DTYPE_BF16)
    enqueue<uint16_t>(a, B, s);
  else
    enqueue<float>(a, B, s);
  return hipGetLastError();
}

}  // namespace fh
