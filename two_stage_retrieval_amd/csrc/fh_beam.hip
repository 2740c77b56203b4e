// Beam search's selection over beams and vocabulary, and the reordering of the
// beams' states.  A candidate (k, t) of a sequence has the score
//   score_k + z_kt - log(sum_u exp(z_ku)),
// and the n candidates with the largest are wanted, in order.  With top_k the
// row's largest logit it is taken as
//   (z_kt - top_k) + (score_k - log(sum_u exp(z_ku - top_k))):
// a row of very large logits (one masked by the type's lowest value throughout) would
// absorb score_k and the logarithm otherwise, and such a beam come before all others.
//
// First launch, per (row, chunk): the sum of exponentials and the largest value
// of each block.  Second, per sequence: a row's chunks are joined, which gives
// both constants of a row, and with them the score of each block's largest
// value.  In the order of scores and, of equal ones, of places, every one of
// the n best candidates lies in one of the n blocks whose largest values are
// the n best: a block outside them has n candidates before all of its own.  So
// n blocks are read again, whatever the values are.  Both times the best n are
// found the same way: the threads hold the entries in sets, the n-th best of the
// sets' best ones is a bound that n entries reach, and the few entries that reach it
// are put in order.
//
// The sums are in fp64: which of two beams' candidates comes first hangs on
// the difference of their sums, and fp32 sums are off by 1e-7, which in a batch
// with thousands of neighbouring candidates a second shows.  (The weights are within
// 4e-14 of theirs.)
#include "fh_device.h"
#include "fh_internal.h"
#include "fh_weights.h"

namespace fh {

namespace {

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / kWave;
constexpr int kBlocks = kBeamChunk / kBeamBlock;   // of a chunk
constexpr double kLog2e = 1.4426950408889634074;

// whether a beam's logits count
__device__ __forceinline__ bool goes_on(const BeamArgs& a, int64_t r) {
  return fabsf(a.scores[r]) < INFINITY && !(a.finished && a.finished[r]);
}

// A wave per (row, chunk); a lane holds 8 values of each block.  A NaN or +inf
// makes the sum NaN; a chunk of -inf alone has sum 0.  256 rows of 128256 in bf16
// take 29 us (66 MB, 12 us at a copy's rate), which the weights' instructions set:
// with two terms less, 1e-10 off, 26; with the fp64 numbers put together by shifts
// instead of converted 30.  Sums that start with the first block to arrive, relative
// to the largest value so far, change nothing.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void beam_rows_kernel(const BeamArgs a) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t id = blockIdx.x * kRowWaves + w, r = id / (uint32_t)a.nchunk;
  if (r >= (uint32_t)a.B * (uint32_t)a.K || !goes_on(a, r)) return;
  const uint8_t* row = a.logits + r * a.l_bytes;
  const int64_t c0 = (int64_t)(id - r * (uint32_t)a.nchunk) * kBeamChunk;
  float x[kBlocks][8], tops[kBlocks];
  bool nan = false;
  if (c0 + kBeamChunk <= a.v) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) load_whole8<T>(row, c0 + i * kBeamBlock + lane * 8, x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      load8<T>(row, c0 + i * kBeamBlock + lane * 8, a.v, -INFINITY, x[i]);
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      m = max3(m, x[i][j], x[i][j + 1]);
      nan |= __builtin_isunordered(x[i][j], x[i][j + 1]);
    }
    tops[i] = wave_max(m);
    top = fmaxf(top, tops[i]);
  }
  if (__ballot(nan)) top = INFINITY;   // (a NaN ends as +inf does)
  double sum = 0.0;
  if (top == INFINITY) {
    sum = NAN;
  } else if (top > -INFINITY) {
    double part[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        part[j & 1] += weight<false>(x[i][j], top, kLog2e, -1020.0 / kLog2e);
    sum = wave_sum_f64(part[0] + part[1]);
  }
  if (lane == 0) {
    a.part_sum[id] = sum;
    reinterpret_cast<float4*>(a.part_top)[id] = make_float4(tops[0], tops[1], tops[2], tops[3]);
  }
}

// A candidate's place in the order: the score as a number that compares as the
// score does (0: none), then the lower index.
struct __align__(16) Place {
  uint32_t hi, lo, at, pad;
};
constexpr Place kNone{0, 0, UINT32_MAX, 0};
// (a 64-bit comparison takes longer than its two halves; no branches)
__device__ __forceinline__ bool before(const Place& x, const Place& y) {
  return (x.hi > y.hi) |
         ((x.hi == y.hi) & ((x.lo > y.lo) | ((x.lo == y.lo) & (x.at < y.at))));
}
__device__ __forceinline__ Place place_of(double score, uint32_t at) {
  const double x = score + 0.0;   // (-0 is 0)
  const uint32_t hi = (uint32_t)__double2hiint(x), lo = (uint32_t)__double2loint(x);
  const uint32_t sign = (uint32_t)((int32_t)hi >> 31);
  return {hi ^ (sign | 0x80000000u), lo ^ sign, at, 0};
}
__device__ __forceinline__ double score_of(const Place& p) {
  const uint32_t sign = (uint32_t)~((int32_t)p.hi >> 31);
  return __hiloint2double((int)(p.hi ^ (sign | 0x80000000u)), (int)(p.lo ^ sign));
}

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / kWave;
constexpr int kMaxOut = 2 * FH_MAX_BEAMS;
constexpr int kMaxSets = 4 * kMaxOut;
constexpr int kList = 4096;        // entries past the first bound,
constexpr int kShort = 512;        // and as many as are put in order
constexpr int kKeep = 8;           // entries of a thread that are taken together

struct SelectShared {
  Place list[kList], list2[kShort], out[kMaxOut];
  uint32_t set[kMaxSets];
  Place best[kSelWaves];
  int count, count2;
  uint32_t least, least2;
};

// The n-th largest of `sets` numbers (a multiple of 64): the waves count, for
// each number, those that come before it (equal ones by their places), and the one
// with n - 1 before it writes *least.
__device__ __forceinline__ void nth_largest(const uint32_t* set, int sets, int n, int w, int lane,
                                            uint32_t* least) {
  uint32_t o[kMaxSets / kWave];
#pragma unroll
  for (int c = 0; c < kMaxSets / kWave; ++c) o[c] = c * kWave < sets ? set[c * kWave + lane] : 0u;
#pragma unroll 4
  for (int i = w; i < sets; i += kSelWaves) {
    const uint32_t mine = (uint32_t)__builtin_amdgcn_readfirstlane((int)set[i]);
    int r = 0;
#pragma unroll
    for (int c = 0; c < kMaxSets / kWave; ++c)
      if (c == 0 || c * kWave < sets) {
        const uint64_t lower = c < i / kWave    ? ~0ull
                               : c == i / kWave ? (1ull << (i % kWave)) - 1
                                                : 0ull;
        r += __builtin_popcountll(__ballot(o[c] > mine) | (__ballot(o[c] == mine) & lower));
      }
    if (r == n - 1 && lane == 0) *least = mine;
  }
}

// The n <= kShort entries of `list` in order; the first ones into s.out.
__device__ __forceinline__ void put_in_order(SelectShared& s, const Place* list, int n, int n_out,
                                             int w, int lane) {
  if (n <= kWave) {
    const Place o = lane < n ? list[lane] : kNone;
#pragma unroll 4
    for (int i = w; i < n; i += kSelWaves) {
      const Place mine = list[i];
      const int r = __builtin_popcountll(__ballot(before(o, mine)));
      if (r < n_out && lane == 0) s.out[r] = mine;
    }
    return;
  }
  for (int i = w; i < n; i += kSelWaves) {
    const Place mine = list[i];
    int r = 0;
    for (int c = 0; c < n; c += kWave)
      r += __builtin_popcountll(__ballot(c + lane < n && before(list[c + lane], mine)));
    if (r < n_out && lane == 0) s.out[r] = mine;
  }
}

// Entries of the threads: fill(b, x) requests kKeep values of batch b (-inf:
// none), place(b, j, x) gives a value's place; the first `used` of each batch count.
template <typename Fill, typename At>
struct Entries {
  Fill fill;
  At place;
  int batches, used;
  Place mine[kKeep];
  __device__ __forceinline__ void request(int b) {
    float x[kKeep];
    fill(b, x);
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      mine[j] = kNone;
      if (j < used && x[j] > -INFINITY) mine[j] = place(b, j, x[j]);
    }
  }
  // Those that may be among the best n, into list (of `room` places): the
  // threads hold the entries in `sets` sets, 4 n at least, and n entries reach the n-th
  // best of the sets' best ones (the upper halves of their places say enough).
  // Returns how many there are, room + 1 if more.
  __device__ __forceinline__ int choose(SelectShared& s, Place* list, int room, int* count,
                                        uint32_t* bound, int n, int w, int lane) {
    int sets = 64;
    while (sets < 4 * n) sets *= 2;
    const int lanes = kSelThreads / sets;   // of a set: 4 to 16 neighbours
    uint32_t best = 0;
    for (int b = 0; b < batches; ++b) {
      request(b);
#pragma unroll
      for (int j = 0; j < kKeep; ++j) best = mine[j].hi > best ? mine[j].hi : best;
    }
    auto up = [&](uint32_t o) { best = o > best ? o : best; };
    up((uint32_t)__builtin_amdgcn_mov_dpp((int)best, 0xB1, 0xf, 0xf, true));  // quad_perm 1 0 3 2
    up((uint32_t)__builtin_amdgcn_mov_dpp((int)best, 0x4E, 0xf, 0xf, true));  // quad_perm 2 3 0 1
    if (lanes >= 8)
      up((uint32_t)__builtin_amdgcn_mov_dpp((int)best, 0x141, 0xf, 0xf, true));  // row_half_mirror
    if (lanes >= 16)
      up((uint32_t)__builtin_amdgcn_mov_dpp((int)best, 0x140, 0xf, 0xf, true));  // row_mirror
    if ((lane & (lanes - 1)) == 0) s.set[(w * kWave + lane) / lanes] = best;
    if (w == 0 && lane == 0) *count = 0;
    __syncthreads();
    nth_largest(s.set, sets, n, w, lane, bound);
    __syncthreads();
    const uint32_t least = *bound > 1u ? *bound : 1u;   // (0: fewer than n sets have an entry)
    for (int b = 0; b < batches; ++b) {
      if (batches > 1) request(b);
#pragma unroll
      for (int j = 0; j < kKeep; ++j)
        if (mine[j].hi >= least) {
          const int to = atomicAdd(count, 1);
          if (to < room) list[to] = mine[j];
        }
    }
    __syncthreads();
    return *count <= room ? *count : room + 1;
  }
  // The best n in order, into s.out, one by one: for entries of which very many
  // are equal in the upper half of their places.  Returns how many there are.
  __device__ __forceinline__ int one_by_one(SelectShared& s, int n, int w, int lane) {
    Place last{UINT32_MAX, UINT32_MAX, 0, 0};
    int found = 0;
    for (; found < n; ++found) {
      Place best = kNone;
      for (int b = 0; b < batches; ++b) {
        request(b);
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
          if (mine[j].hi && before(last, mine[j]) && before(mine[j], best)) best = mine[j];
      }
#pragma unroll
      for (int m = 1; m < kWave; m *= 2) {
        const Place o{(uint32_t)__shfl_xor((int)best.hi, m), (uint32_t)__shfl_xor((int)best.lo, m),
                      (uint32_t)__shfl_xor((int)best.at, m), 0};
        if (before(o, best)) best = o;
      }
      __syncthreads();
      if (lane == 0) s.best[w] = best;
      __syncthreads();
      best = kNone;
      for (int i = 0; i < kSelWaves; ++i)
        if (before(s.best[i], best)) best = s.best[i];
      if (!best.hi) break;
      last = best;
      if (w == 0 && lane == 0) s.out[found] = best;
    }
    return found;
  }
};

// The best n of the entries in order, into s.out; returns how many there are (n
// at most).  All threads; s.out may be read until the next call has put its own there.
template <typename Fill, typename At>
__device__ __forceinline__ int best_of(SelectShared& s, Fill fill, At place, int batches, int used,
                                       int n, int w, int lane) {
  Entries<Fill, At> all{fill, place, batches, used, {}};
  int count = all.choose(s, s.list, kList, &s.count, &s.least, n, w, lane);
  const Place* list = s.list;
  if (count > kShort && count <= kList) {   // once more, among those
    const int some = count, tid = w * kWave + lane;
    auto again = [&](int, float* x) {
#pragma unroll
      for (int j = 0; j < kKeep; ++j) x[j] = j * kSelThreads + tid < some ? 0.0f : -INFINITY;
    };
    auto at = [&](int, int j, float) { return s.list[j * kSelThreads + tid]; };
    Entries<decltype(again), decltype(at)> few{again, at, 1, kList / kSelThreads, {}};
    count = few.choose(s, s.list2, kShort, &s.count2, &s.least2, n, w, lane);
    list = s.list2;
    if (count > kShort) {
      count = few.one_by_one(s, n, w, lane);
      __syncthreads();
      return count;
    }
  } else if (count > kList) {
    count = all.one_by_one(s, n, w, lane);
    __syncthreads();
    return count;
  }
  put_in_order(s, list, count, n, w, lane);
  __syncthreads();
  return count < n ? count : n;
}

// One workgroup per sequence.  A chain of dependent steps sets its time, 8 us for 4
// beams of 128256 and 8 candidates: the rows' sums (1.5 us), blocks (2.5), values (3,
// of which 1.2 to read them), and the launch; 9 for 64 sequences, 18 for 16 beams and
// 32 candidates.
template <typename T>
__global__ __launch_bounds__(kSelThreads) void beam_select_kernel(const BeamArgs a) {
  __shared__ SelectShared s;
  struct __align__(16) Row {
    double top, rest;   // its largest logit; its score less the sum's logarithm
    __device__ __forceinline__ double score(float x) const { return ((double)x - top) + rest; }
  };
  __shared__ Row s_row[FH_MAX_BEAMS];
  __shared__ uint8_t s_kind[FH_MAX_BEAMS];  // 0 no candidate, 1 its logits, 2 has ended
  struct Block {
    Row row;
    int64_t first;   // its first token
    int beam, kind;
  };
  __shared__ Block s_block[kMaxOut];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t r0 = (int64_t)blockIdx.x * a.K;
  const uint32_t nblk = a.nchunk * kBlocks;
  const int entries = a.K * (int)nblk;
  const float* part_top = a.part_top + r0 * nblk;
  auto request_tops = [&](int b, float* x) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      const int i = (b * kKeep + j) * kSelThreads + tid;
      x[j] = -INFINITY;
      if (i < entries) x[j] = part_top[i];
    }
  };
  float tops[kKeep];   // on their way while the rows are joined
  request_tops(0, tops);
  for (int k = w; k < a.K; k += kSelWaves) {
    const int64_t r = r0 + k;
    const double* sum = a.part_sum + r * a.nchunk;
    const float4* of = reinterpret_cast<const float4*>(a.part_top) + r * a.nchunk;
    const float score = a.scores[r];
    const bool ended = a.finished && a.finished[r];
    // (what is not written is read here too, and not used)
    float top = -INFINITY;
    double total = 0.0;
    for (int c0 = 0; c0 < a.nchunk; c0 += kWave) {
      const int c = c0 + lane;
      float m = -INFINITY;
      double p = 0.0;
      if (c < a.nchunk) {
        const float4 t = of[c];
        m = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w));
        p = sum[c];
      }
      const float up = fmaxf(top, wave_max(m));
      if (up > -INFINITY) {
        if (top > -INFINITY) total *= weight(top, up, kLog2e);
        total += m == -INFINITY && p == 0.0 ? 0.0 : p * weight(m, up, kLog2e);
      } else {
        total += p;   // 0 or NaN
      }
      top = up;
    }
    total = wave_sum_f64(total);
    if (lane == 0) {
      const bool there = fabsf(score) < INFINITY;
      s_kind[k] = (uint8_t)(!there ? 0 : ended ? 2 : total > 0.0 ? 1 : 0);   // (NaN: none)
      s_row[k] = ended ? Row{0.0, (double)score} : Row{(double)top, (double)score - log(total)};
    }
  }
  __syncthreads();

  // the blocks: an ended beam's first one stands for its only candidate
  auto beam_of = [&](int i) { return (int)__umulhi((uint32_t)i, a.by_nblk); };
  const int per = (entries + kSelThreads - 1) / kSelThreads;   // of a thread
  const int blocks = best_of(
      s,
      [&](int b, float* x) {
        if (b == 0) {
#pragma unroll
          for (int j = 0; j < kKeep; ++j) x[j] = tops[j];
        } else {
          request_tops(b, x);
        }
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
          const int i = (b * kKeep + j) * kSelThreads + tid;
          if (i < entries) {
            const int k = beam_of(i), kind = s_kind[k];
            x[j] = kind == 1 ? x[j] : kind == 2 && i == k * (int)nblk ? 0.0f : -INFINITY;
          }
        }
      },
      [&](int b, int j, float x) {
        const int i = (b * kKeep + j) * kSelThreads + tid;
        return place_of(s_row[beam_of(i)].score(x), (uint32_t)i);
      },
      (per + kKeep - 1) / kKeep, per < kKeep ? per : kKeep, a.n_out, w, lane);
  if (tid < blocks) {
    const int i = (int)s.out[tid].at, k = beam_of(i);
    s_block[tid] = Block{s_row[k], (int64_t)(i - k * (int)nblk) * kBeamBlock, k, s_kind[k]};
  }
  __syncthreads();

  // their values: a block a wave, 8 in a row a lane
  static_assert(kBeamBlock == kWave * kKeep, "a block a wave");
  Block now{{0.0, 0.0}, 0, 0, 0};
  const int found = best_of(
      s,
      [&](int b, float* x) {
        const int at = b * kSelWaves + w;
        now = s_block[at < blocks ? at : 0];
        if (at >= blocks || now.kind == 2) {
#pragma unroll
          for (int j = 0; j < kKeep; ++j) x[j] = -INFINITY;
          if (at < blocks && lane == 0) x[0] = 0.0f;
        } else {
          load8<T>(a.logits + (r0 + now.beam) * a.l_bytes, now.first + lane * kKeep, a.v, -INFINITY,
                   x);
        }
      },
      [&](int, int j, float x) {
        const uint32_t t =
            now.kind == 2 ? (uint32_t)a.pad_token : (uint32_t)now.first + lane * kKeep + j;
        return place_of(now.row.score(x), (uint32_t)(now.beam * a.v) + t);
      },
      (blocks + kSelWaves - 1) / kSelWaves, kKeep, a.n_out, w, lane);
  if (tid < a.n_out) {
    const int64_t o = (int64_t)blockIdx.x * a.n_out + tid;
    const bool there = tid < found;
    const Place p = s.out[there ? tid : 0];
    const int k = there ? (int)(p.at / (uint32_t)a.v) : 0;
    const int t = (int)(p.at - (uint32_t)k * (uint32_t)a.v);
    a.out_scores[o] = there ? (float)score_of(p) : -INFINITY;
    a.out_parents[o] = there ? k : -1;
    a.out_tokens[o] = there ? t : -1;
    if (a.out_finished) a.out_finished[o] = there && (s_kind[k] == 2 || t == a.eos_token) ? 1 : 0;
  }
}

template <typename T>
void enqueue_select(const BeamArgs& a, hipStream_t s) {
  const int64_t parts = (int64_t)a.B * a.K * a.nchunk;
  hipLaunchKernelGGL(beam_rows_kernel<T>, dim3((unsigned)((parts + kRowWaves - 1) / kRowWaves)),
                     dim3(kRowThreads), 0, s, a);
  hipLaunchKernelGGL(beam_select_kernel<T>, dim3((unsigned)a.B), dim3(kSelThreads), 0, s, a);
}

// ---------------------------------------------------------------------------
// Reordering.  A thread holds the same bytes of every beam of a sequence that
// changes, so that all are read before one is written and no thread waits for
// another, in place as well.  Bound by memory: of 4 beams 2 change, 2.1 GB read and
// written past the caches in 361 us (5.8 TB/s; two units of 16 bytes a thread and beam,
// with one 541, with four 382, without the non-temporal hints 401).
// ---------------------------------------------------------------------------
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
constexpr int kMoveThreads = 256;

// grid: pieces of kUnits * 256 W along the positions, (outer, inner), sequences;
// what a launch has no room for comes in a loop
template <typename W, int kBeams, int kUnits>
__global__ __launch_bounds__(kMoveThreads) void beam_reorder_kernel(const ReorderArgs a,
                                                                    int64_t rows) {
  constexpr int kStep = kMoveThreads * (int)sizeof(W), kPer = kUnits * kStep;
  const bool in_place = a.src == a.dst;
  for (int s = blockIdx.z; s < a.B; s += gridDim.z) {
    int64_t n = a.positions;
    if (a.lengths) {
      const int64_t len = a.lengths[s];
      n = len < 0 ? 0 : len < n ? len : n;
    }
    n *= a.pos_bytes;
    int from[kBeams];   // (-1: nothing to do)
#pragma unroll
    for (int j = 0; j < kBeams; ++j) {
      from[j] = -1;
      if (j < a.K) {
        const int p = a.parents[(int64_t)s * a.K + j];
        from[j] = p >= 0 && p < a.K ? p : j;
        if (in_place && from[j] == j) from[j] = -1;
      }
    }
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
      const int64_t o = a.inner > 1 ? row / a.inner : row, i = a.inner > 1 ? row % a.inner : 0;
      const int64_t base =
          o * a.outer_stride + (int64_t)s * a.K * a.beam_stride + i * a.inner_stride;
      for (int64_t first = blockIdx.x * (int64_t)kPer; first < n;
           first += gridDim.x * (int64_t)kPer) {
        const int64_t at = first + threadIdx.x * (int)sizeof(W);
        const uint8_t* src = a.src + base + at;
        uint8_t* dst = a.dst + base + at;
        W x[kBeams][kUnits];
#pragma unroll
        for (int j = 0; j < kBeams; ++j)
          if (from[j] >= 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              if (at + u * kStep < n)
                x[j][u] = __builtin_nontemporal_load(
                    reinterpret_cast<const W*>(src + from[j] * a.beam_stride + u * kStep));
          }
#pragma unroll
        for (int j = 0; j < kBeams; ++j)
          if (from[j] >= 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              if (at + u * kStep < n)
                __builtin_nontemporal_store(
                    x[j][u], reinterpret_cast<W*>(dst + j * a.beam_stride + u * kStep));
          }
      }
    }
  }
}

template <typename W, int kBeams, int kUnits>
void enqueue_move(const ReorderArgs& a, hipStream_t s) {
  constexpr int64_t kPer = (int64_t)kUnits * kMoveThreads * sizeof(W);
  int64_t pieces = (a.positions * a.pos_bytes + kPer - 1) / kPer;
  const int64_t rows = a.outer * a.inner;
  // With lengths of their own the sequences leave many pieces empty, which cost a
  // workgroup each: then 8192 workgroups walk over the pieces (lengths spread over
  // [60, 1000] of 1000: 234 us, with a workgroup for every piece 279; all of them
  // 1000: 415 and 361).
  if (a.lengths) {
    const int64_t some = 8192 / (rows < 8192 ? rows : 8192) / (a.B < 8192 ? a.B : 8192);
    pieces = pieces < some ? pieces : some > 1 ? some : 1;
  }
  const dim3 grid((unsigned)(pieces < (1 << 20) ? pieces : 1 << 20),
                  (unsigned)(rows < 65535 ? rows : 65535), (unsigned)(a.B < 65535 ? a.B : 65535));
  hipLaunchKernelGGL((beam_reorder_kernel<W, kBeams, kUnits>), grid, dim3(kMoveThreads), 0, s, a,
                     rows);
}

template <typename W>
void enqueue_reorder(const ReorderArgs& a, hipStream_t s) {
  if (a.K <= 4)
    enqueue_move<W, 4, 2>(a, s);
  else if (a.K <= 8)
    enqueue_move<W, 8, 2>(a, s);
  else if (a.K <= 16)
    enqueue_move<W, 16, 1>(a, s);
  else
    enqueue_move<W, FH_MAX_BEAMS, 1>(a, s);
}

}  // namespace

hipError_t launch_beam_select(const BeamArgs& a, int dtype, hipStream_t s) {
  if (dtype == FH_DTYPE_BF16)
    enqueue_select<uint16_t>(a, s);
  else
    enqueue_select<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
  const uint64_t bits = (uint64_t)(uintptr_t)a.src | (uint64_t)(uintptr_t)a.dst |
                        (uint64_t)a.outer_stride | (uint64_t)a.beam_stride |
                        (uint64_t)a.inner_stride | (uint64_t)a.pos_bytes;
  if (bits % 16 == 0)
    enqueue_reorder<v4u>(a, s);
  else if (bits % 4 == 0)
    enqueue_reorder<uint32_t>(a, s);
  else
    enqueue_reorder<uint8_t>(a, s);
  return hipGetLastError();
}

}  // namespace fh
