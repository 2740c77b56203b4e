// Logits of the 8-bit dense head:
//   z[m, t] = sum_g hs[m, g] es[t / 128, g] sum_{k in block g} h8[m, k] e8[t, k]
// over e4m3 codes, one fp32 scale per 128 columns of a row of h and per
// 128 x 128 block of E.  The products of a block of 128 columns are summed by
// the matrix cores; its fp32 result is then scaled and added to the fp32
// accumulator, since the scales change from block to block.
#include "fh_device.h"
#include "fh_host.h"
#include "fh_internal.h"

namespace fh {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
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

// A lane's 32 bytes of a 16-row operand's block, as bf16 values, as the matrix
// instruction takes them: lane l gives bytes of row l % 16 (any order of the
// columns that both operands share).
//
// The 8-bit matrix instruction would take the codes themselves at twice the
// rate, but cuts products short: within each group of 8 it drops the bits below
// 2^-13 of the group's largest product (measured; 4.5e-5 of the result on codes
// spread over the whole format, against 3e-8 for the bf16 instruction).  The
// sums are held to 32 bits here, for every number of rows and type of output.
struct Frag {
  v8bf x[4];
  __device__ __forceinline__ void set(v4i lo, v4i hi) {
    x[0] = to_bf16(lo[0], lo[1]);
    x[1] = to_bf16(lo[2], lo[3]);
    x[2] = to_bf16(hi[0], hi[1]);
    x[3] = to_bf16(hi[2], hi[3]);
  }
};

// D[i, j] = sum over a block's columns of A[i, :] . B[j, :]; lane l receives
// rows 4 (l / 16) + 0..3 of column l % 16
__device__ __forceinline__ v4f mfma128(const Frag& a, const Frag& b) {
  v4f c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x[i], b.x[i], c, 0, 0, 0);
  return c;
}

// 16 bytes of a row at column k, zero past its end (d is a multiple of 16)
__device__ __forceinline__ v4i chunk(const uint8_t* row, int k, int d) {
  if (k < d) return *reinterpret_cast<const v4i*>(row + k);
  return v4i{0, 0, 0, 0};
}

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4u bf16_pair(v4f a, v4f b) {
  return __builtin_bit_cast(v4u, __builtin_shufflevector(__builtin_convertvector(a, v4bf),
                                                         __builtin_convertvector(b, v4bf), 0, 1, 2,
                                                         3, 4, 5, 6, 7));
}

// Column of result i (0 .. 3) of a lane's tile j in a run of 16 NT columns,
// less i: each store instruction writes 64 bytes in a row (16 columns of
// fp32, or of two tiles' 32 of bf16).  Result row r = 4 q + i of tile j is
// row run_at(j, q) + i of E.
template <typename TO, int NT>
__device__ __forceinline__ int run_at(int j, int q) {
  if constexpr (sizeof(TO) == 2 && NT > 1) return 32 * (j >> 1) + 8 * q + 4 * (j & 1);
  return 16 * j + 4 * q;
}

// A lane's results of row m, columns n + run_at(j, q) + 0..3.
template <typename TO, int NT>
__device__ __forceinline__ void store_run(const Logits8Args& a, int m, int64_t n, int q,
                                          const v4f* x) {
  TO* row = reinterpret_cast<TO*>(a.out) + (int64_t)m * a.ldo;
  constexpr int P = sizeof(TO) == 2 && NT > 1 ? 2 : 1;   // tiles per store
#pragma unroll
  for (int j = 0; j < NT; j += P) {
    const int64_t t = n + run_at<TO, NT>(j, q);
    TO y[4 * P];
#pragma unroll
    for (int i = 0; i < 4 * P; ++i) {
      const float z = x[j + i / 4][i % 4];
      if constexpr (sizeof(TO) == 4) y[i] = z;
      else y[i] = __builtin_bit_cast(uint16_t, (__bf16)z);
    }
    if (t + 4 * P <= a.v) {
      typedef uint32_t words __attribute__((ext_vector_type(P * sizeof(TO))));
      words u;
      __builtin_memcpy(&u, y, sizeof(u));
      *reinterpret_cast<words*>(row + t) = u;
    } else {
#pragma unroll
      for (int i = 0; i < 4 * P; ++i)
        if (t + i < a.v) row[t + i] = y[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: kBM rows of h by kBN of E per workgroup of 8 waves, each wave kBM / 2
// by kBN / 4.  Blocks of 128 columns go from memory to LDS without passing
// registers (two buffers: the next block's loads run under the present block's
// products).
// ---------------------------------------------------------------------------
// LDS rows are 128 bytes: eight 16-byte slots.  Chunk k of row r is held in
// slot k ^ key(r), so that the eight lanes that read one chunk of eight rows
// at a time touch eight different slots.
__device__ __forceinline__ int key_h(int r) { return r & 7; }
// (tiles of E take rows as run_at says: 8 lanes read rows of which bits 0, 1
// and 3 differ, or 0 to 2)
template <typename TO>
__device__ __forceinline__ int key_e(int r) {
  return sizeof(TO) == 2 ? (r & 3) | ((r >> 1) & 4) : r & 7;
}

// Memory to LDS: 16 (or 4) bytes a lane from base + off to the wave's LDS
// address, lane after lane.  Written as instructions because the compiler,
// which cannot tell the two buffers apart, would wait for the next block's
// loads before it reads the present one; the waits are load_lds_wait's.  They
// write no register, so nothing can be taken for written too early.
__device__ __forceinline__ uint32_t lds_address(void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)p;
}
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
// Waits until at most n of the wave's memory operations, the last ones, are
// open (they end in the order in which they were issued, stores among them).
template <int n>
__device__ __forceinline__ void load_lds_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "i"(n) : "memory");
}

// One workgroup per compute unit takes tile after tile.  The rows of E of block
// s + 2 are requested during block s, as soon as every wave has its operands
// of E in registers; those of h (which stay in the die's cache) one block
// ahead.  This goes on over the ends of tiles, and a tile's stores are behind
// the loads of the next one's first block, so that neither stands alone.
//
// 2048 x 128256 x 2048 to bf16 takes 1012 to 1054 us (1.02 to 1.06 PFLOP/s; a
// library's bf16 product of these sizes, without the scales and with E already in
// bf16, 943), to fp32 1080.  The matrix instructions fill 489 us at 2.1 GHz (43 %
// busy); between them are the conversions of both operands, the LDS reads and
// the sums.
constexpr int kTileGroups = kLogits8Groups;

template <int kBM, int kBN, typename TO>
__global__ __launch_bounds__(512, 2) void logits8_tiles_kernel(const Logits8Args a) {
  constexpr int MT = kBM / 32;   // 16-row tiles of h per wave
  constexpr int NT = kBN / 64;   // and of E
  constexpr int kStores = MT * NT / (sizeof(TO) == 2 ? 2 : 1);   // of a wave's results
  __shared__ __align__(128) uint8_t s_e[2][kBN * 128];
  __shared__ __align__(128) uint8_t s_h[2][kBM * 128];
  __shared__ __align__(128) float s_hs[2][kBM];
  __shared__ __align__(128) float s_es[2][kWave];  // the tile's two blocks of E, then copies
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w >> 2, wn = w & 3;

  // Workgroups are dealt to the 8 compute dies in turn: each die has a run of
  // tiles, up to 4 of h under one of E, so that it reads its rows of E into
  // its cache once for four tiles and keeps the rows of h there.
  const unsigned mt = (unsigned)(a.rows + kBM - 1) / kBM, nt = (unsigned)((a.v + kBN - 1) / kBN);
  const unsigned tiles = mt * nt, per = (tiles + 7) / 8;
  const unsigned last = min(tiles, (blockIdx.x % 8 + 1) * per);
  unsigned tile = blockIdx.x % 8 * per + blockIdx.x / 8;
  if (tile >= last) return;

  // loads: each wave fills 8 rows of 8 slots at a time; scales: wave w < kBM /
  // 64 those of 64 rows of h, the last wave E's
  const int lr = lane >> 3, slot = lane & 7;
  const int e_k = 16 * (slot ^ key_e<TO>(w * 8 + lr)), h_k = 16 * (slot ^ key_h(lr));
  const uint32_t l_e = lds_address(s_e) + w * 1024, l_h = lds_address(s_h) + w * 1024;
  const uint32_t l_s = w == 7 ? lds_address(s_es) : lds_address(s_hs) + w * 256;
  auto place = [&](unsigned tile, int* m0, int64_t* n0) {
    const unsigned group = tile / (4 * nt), gm = min(4u, mt - group * 4);
    const unsigned in = tile - group * 4 * nt;
    *m0 = (int)(group * 4 + in % gm) * kBM;
    *n0 = (int64_t)(in / gm) * kBN;
  };
  // The two streams of loads: the tile and block that comes next, and where
  // it is.  A chunk past a row's end: the row's first bytes instead, which the
  // products leave out.
  const int G = (a.d + 127) / 128;
  unsigned e_tile = tile, h_tile = tile;
  int e_kb = 0, h_kb = 0;
  const uint8_t *e_base, *h_base;
  const float* s_base;
  uint32_t e_off[kBN / 64], h_off[kBM / 64], s_off;
  auto e_at = [&]() {
    int m0;
    int64_t n0;
    place(e_tile, &m0, &n0);
    e_base = a.E8 + n0 * a.lde;
    const int e_last = (int)min(a.v - 1 - n0, (int64_t)kBN);
#pragma unroll
    for (int i = 0; i < kBN / 64; ++i)
      e_off[i] = (uint32_t)min(i * 64 + w * 8 + lr, e_last) * (uint32_t)a.lde;
  };
  auto h_at = [&]() {
    int m0;
    int64_t n0;
    place(h_tile, &m0, &n0);
    h_base = a.h8 + (int64_t)m0 * a.ldh;
    const int h_last = a.rows - 1 - m0;
#pragma unroll
    for (int i = 0; i < kBM / 64; ++i)
      h_off[i] = (uint32_t)min(i * 64 + w * 8 + lr, h_last) * (uint32_t)a.ldh;
    const bool two = lane > 0 && n0 / 128 < (a.v - 1) / 128;
    s_base = w == 7 ? a.E_scale + n0 / 128 * a.ldes : a.h_scale + (int64_t)m0 * a.lds;
    s_off = w == 7 ? (two ? (uint32_t)a.ldes * 4 : 0u)
                   : (uint32_t)min(tid, h_last) * (uint32_t)a.lds * 4;
  };
  // kELoads of a wave; false when there is no more
  constexpr int kELoads = kBN / 64;
  auto load_e = [&](int st) {
    if (e_tile >= last) return false;
    const int k0 = e_kb * 128;
    const bool whole = k0 + 128 <= a.d;
    const uint8_t* base = whole ? e_base + k0 : e_base;
    const uint32_t k = whole ? e_k : k0 + e_k < a.d ? k0 + e_k : 0;
#pragma unroll
    for (int i = 0; i < kELoads; ++i)
      load_lds16(base, e_off[i] + k, l_e + st * (kBN * 128) + i * 8192);
    if (++e_kb == G) {
      e_kb = 0;
      e_tile += kTileGroups / 8;
      if (e_tile < last) e_at();
    }
    return true;
  };
  auto load_h = [&](int st) {
    if (h_tile >= last) return;
    const int k0 = h_kb * 128;
    const bool whole = k0 + 128 <= a.d;
    const uint8_t* base = whole ? h_base + k0 : h_base;
    const uint32_t k = whole ? h_k : k0 + h_k < a.d ? k0 + h_k : 0;
#pragma unroll
    for (int i = 0; i < kBM / 64; ++i)
      load_lds16(base, h_off[i] + k, l_h + st * (kBM * 128) + i * 8192);
    if (w < kBM / 64)
      load_lds4(s_base + h_kb, s_off, l_s + st * (kBM * 4));
    else if (w == 7)
      load_lds4(s_base + h_kb, s_off, l_s + st * (kWave * 4));
    if (++h_kb == G) {
      h_kb = 0;
      h_tile += kTileGroups / 8;
      if (h_tile < last) h_at();
    }
  };

  // where the lane's operands are in LDS: row and byte of the first chunk (the
  // second is four slots on), and the rows between tiles
  const int e_row = wn * (kBN / 4) + run_at<TO, NT>(0, c >> 2) + (c & 3);
  const int e_slot = 16 * (q ^ key_e<TO>(e_row));
  const int h_row = wm * (kBM / 2) + c, h_slot = 16 * (q ^ key_h(c));
  // the last block of a row that is not whole: h counts as zero past its end
  auto cut = [&](int st) {
    const int from = (a.d % 128) / 16;
    for (int i = tid; i < kBM * 8; i += 512)
      if ((i & 7) >= from)
        *reinterpret_cast<v4i*>(s_h[st] + (i >> 3) * 128 + 16 * ((i & 7) ^ key_h(i >> 3))) =
            v4i{0, 0, 0, 0};
    __syncthreads();
  };

  v4f acc[MT][NT];
  auto clear = [&]() {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // Stores the wave's part of the tile at m, n, which ends before the last
  // column.  A row that does not exist goes to an offset past the resource's
  // end, which drops the store: there are always kStores of them.
  auto store = [&](int m, int64_t n) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<uint8_t*>(a.out) + ((int64_t)m * a.ldo + n) * sizeof(TO), 0, 0x7FFFFFFF,
        0x00027000);
    if constexpr (sizeof(TO) == 2 && NT == 4) {
      // Eight rows of 128 bytes a store instead of sixteen of 64: lane c of a
      // row's first 8 gives away its second half and takes lane c + 8's
      // first (16 us less at 2048 x 128256 x 2048).
      const bool up = c >= 8;
      const uint32_t lane_off = (uint32_t)((c & 7) * a.ldo + 8 * q + (up ? 32 : 0)) * 2;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const v4u y[2] = {bf16_pair(acc[t][0], acc[t][1]), bf16_pair(acc[t][2], acc[t][3])};
        v4u z;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // row_ror:8: the lane 8 on in its row of 16
          z[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(up ? y[0][i] : y[1][i]), 0x128,
                                                       0xf, 0xf, false);
#pragma unroll
        for (int o = 0; o < 2; ++o) {  // rows 0..7, then 8..15 of the 16
          const v4u x = (o == 1) == up ? y[o] : z;
          const uint32_t off =
              m + t * 16 + o * 8 + (c & 7) < a.rows
                  ? lane_off + (uint32_t)((t * 16 + o * 8) * a.ldo) * 2
                  : 0x80000000u;
          __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, (int)off, 0, 0);
        }
      }
    } else {
      constexpr int P = sizeof(TO) == 2 ? 2 : 1;   // tiles per store
      const uint32_t lane_off = (uint32_t)(c * a.ldo + run_at<TO, NT>(0, q)) * sizeof(TO);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint32_t off = m + t * 16 + c < a.rows
                                 ? lane_off + (uint32_t)(t * 16 * a.ldo) * sizeof(TO)
                                 : 0x80000000u;
#pragma unroll
        for (int j = 0; j < NT; j += P) {
          v4u x;
          if constexpr (P == 2)
            x = bf16_pair(acc[t][j], acc[t][j + 1]);
          else
            x = __builtin_bit_cast(v4u, acc[t][j]);
          __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, (int)(off + 64 * (j / P)), 0, 0);
        }
      }
    }
  };

  // adds the products of the block in buffer st; true if loads of E were made
  auto block = [&](int st) {
    bool more = false;
    const float s_e_scale = s_es[st][wn * (kBN / 4) / 128];
    Frag e[NT];
    const uint8_t* pe = s_e[st] + e_row * 128;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      e[j].set(*reinterpret_cast<const v4i*>(pe + run_at<TO, NT>(j, 0) * 128 + e_slot),
               *reinterpret_cast<const v4i*>(pe + run_at<TO, NT>(j, 0) * 128 + (e_slot ^ 64)));
    const uint8_t* ph = s_h[st] + h_row * 128;
    v4i lo, hi;
    float s;
    auto read_h = [&](int t) {
      lo = *reinterpret_cast<const v4i*>(ph + t * 2048 + h_slot);
      hi = *reinterpret_cast<const v4i*>(ph + t * 2048 + (h_slot ^ 64));
      s = s_hs[st][h_row + t * 16];
    };
    // The sums are taken here: the compiler would gather them behind the next
    // branch otherwise, and hold every product until then.
    auto pin = [&]() {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[t][j]));
    };
    v4f x[NT];
    float xs = 0.0f;
    auto add = [&](int t, int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(x[j][i], xs, acc[t][j][i]);
    };
    read_h(0);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      Frag h;
      h.set(lo, hi);
      const float x_scale = s * s_e_scale;
      if (t + 1 < MT) read_h(t + 1);
      // The products of this tile run while the last one's are added, four
      // matrix instructions (64 cycles) to four sums (16).
      v4f y[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        y[j] = mfma128(e[j], h);
        if (t > 0) add(t - 1, j);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) x[j] = y[j];
      xs = x_scale;
      // (reads stay one tile ahead: all at once they would not fit the registers)
      __builtin_amdgcn_sched_barrier(0);
      if (t == (MT > 2 ? 1 : 0)) {
        // E's operands are in every wave's registers: the buffer is free
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        more = load_e(st);
        pin();
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) add(MT - 1, j);
    pin();
    return more;
  };

  e_at();
  h_at();
  load_e(0);
  load_h(0);
  load_e(1);
  load_lds_wait<0>();
  __syncthreads();
  if (G == 1 && a.d % 128) cut(0);
  for (int st = 0; tile < last; tile += kTileGroups / 8) {
    int m0;
    int64_t n0;
    place(tile, &m0, &n0);
    const int m1 = m0 + wm * (kBM / 2);
    const int64_t n1 = n0 + wn * (kBN / 4);
    clear();
    for (int kb = 0; kb + 1 < G; ++kb) {
      load_h(st ^ 1);
      if (block(st))
        load_lds_wait<kELoads>();  // all but E's of the block after the next
      else
        load_lds_wait<0>();
      __syncthreads();
      st ^= 1;
      if (kb + 2 == G && a.d % 128) cut(st);
    }
    load_h(st ^ 1);
    const bool more = block(st);
    if (n0 + kBN <= a.v) {
      store(m1, n1);
      if (more)
        load_lds_wait<kELoads + kStores>();
      else
        load_lds_wait<kStores>();
    } else {  // the last column cuts some stores: value by value
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (m1 + t * 16 + c < a.rows) store_run<TO, NT>(a, m1 + t * 16 + c, n1, q, acc[t]);
      load_lds_wait<0>();
    }
    __syncthreads();
    st ^= 1;
    if (G == 1 && a.d % 128 && tile + kTileGroups / 8 < last) cut(st);
  }
}

// ---------------------------------------------------------------------------
// Few rows, or few tiles: four waves share 16 MT rows of h and 16 NT of E,
// take every fourth block of columns each, and add their sums through LDS in
// wave order.  Operands go straight to registers, the next block's while the
// present one is multiplied.  Bound by reading E: 1 x 128256 x 2048 takes 44.5
// us (5.9 TB/s; a plain read of 1 GiB reaches 5.5, part of E stays in the
// memory-side cache).
// ---------------------------------------------------------------------------
constexpr int kSplit = kLogits8Split;

template <int MT, int NT, typename TO>
__global__ __launch_bounds__(256, 2) void logits8_rows_kernel(const Logits8Args a) {
  const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  const int m0 = blockIdx.y * (16 * MT);
  const uint8_t* e[NT];
  const uint8_t* h[MT];
  const float* hs[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + run_at<TO, NT>(j, c >> 2) + (c & 3);
    e[j] = a.E8 + (n < a.v ? n : a.v - 1) * a.lde;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + c < a.rows ? m0 + 16 * t + c : a.rows - 1;
    h[t] = a.h8 + (int64_t)m * a.ldh;
    hs[t] = a.h_scale + (int64_t)m * a.lds;
  }
  const float* es = a.E_scale + (n0 / 128) * a.ldes;
  v4f acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int G = (a.d + 127) / 128;
  // the next block's rows are on their way while this one is multiplied
  struct Raw { v4i lo, hi; } re[NT], rh[MT];
  float s[MT];
  auto load = [&](int kb) {
    const int k = kb * 128 + 16 * q;
#pragma unroll
    for (int j = 0; j < NT; ++j) re[j] = Raw{chunk(e[j], k, a.d), chunk(e[j], k + 64, a.d)};
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      rh[t] = Raw{chunk(h[t], k, a.d), chunk(h[t], k + 64, a.d)};
      s[t] = hs[t][kb] * es[kb];
    }
  };
  int kb = w;
  if (kb < G) load(kb);
  for (; kb < G; kb += kSplit) {
    Frag ef[NT], hf[MT];
    float sc[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) ef[j].set(re[j].lo, re[j].hi);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      hf[t].set(rh[t].lo, rh[t].hi);
      sc[t] = s[t];
    }
    if (kb + kSplit < G) load(kb + kSplit);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v4f x = mfma128(ef[j], hf[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(x[i], sc[t], acc[t][j][i]);
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
    if (m < a.rows) store_run<TO, NT>(a, m, n0, q, acc[t]);
  }
}

template <int MT, int NT, typename TO>
void enqueue_rows(const Logits8Args& a, hipStream_t s) {
  hipLaunchKernelGGL((logits8_rows_kernel<MT, NT, TO>),
                     dim3((unsigned)((a.v + 16 * NT - 1) / (16 * NT)),
                          (unsigned)((a.rows + 16 * MT - 1) / (16 * MT))),
                     dim3(256), 0, s, a);
}

template <int kBM, int kBN, typename TO>
void enqueue_tiles(const Logits8Args& a, hipStream_t s) {
  hipLaunchKernelGGL((logits8_tiles_kernel<kBM, kBN, TO>), dim3(kTileGroups), dim3(512), 0, s, a);
}

template <typename TO>
void enqueue(const Logits8Args& a, hipStream_t s) {
  const Logits8Plan p = plan_logits8(a.rows, a.v, a.d, a.ldo, sizeof(TO));
  if (p.tiles) {
    switch (p.bm * 1000 + p.bn) {
      case 64128: enqueue_tiles<64, 128, TO>(a, s); break;
      case 128128: enqueue_tiles<128, 128, TO>(a, s); break;
      case 64256: enqueue_tiles<64, 256, TO>(a, s); break;
      case 128256: enqueue_tiles<128, 256, TO>(a, s); break;
    }
    return;
  }
  switch (p.bm * 1000 + p.bn) {
    case 16016: enqueue_rows<1, 1, TO>(a, s); break;
    case 16032: enqueue_rows<1, 2, TO>(a, s); break;
    case 16064: enqueue_rows<1, 4, TO>(a, s); break;
    case 32064: enqueue_rows<2, 4, TO>(a, s); break;
  }
}

}  // namespace

hipError_t launch_logits8(const Logits8Args& a, int out_dtype, hipStream_t s) {
  if (out_dtype == FH_DTYPE_BF16)
    enqueue<uint16_t>(a, s);
  else
    enqueue<float>(a, s);
  return hipGetLastError();
}

}  // namespace fh
