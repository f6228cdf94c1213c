// lora_linear.hip - low-rank adapters of many requests beside a shared projection
// (skinny_lora_linear), on MI355X (gfx950).

#include <hip/hip_runtime.h>

#include "host_util.h"
#include "skinny_gemm.h"

namespace {

using skinny_host::DeviceInfo;
using skinny_host::Range;
using skinny_host::aligned;
using skinny_host::device_info;
using skinny_host::overlap;
using skinny_host::range_of;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // y's rows of an odd width
typedef u32x4 u32x4_dword __attribute__((aligned(4)));
typedef unsigned u32x3 __attribute__((ext_vector_type(3)));
typedef u32x3 u32x3_dword __attribute__((aligned(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// y[t] = base[t] + scale B (A x[t]) on the matrix cores, v_mfma_f32_16x16x32_bf16,
// fp32 sums: A x with A = 16 ranks and B = 16 rows, so that lane (c, g) ends with four
// neighbouring ranks of row c; then, B's columns for A and the rows' A x for B, with
// neighbouring columns of one row of y.  Between the two products A x, an fp32 number of
// 24 bits, is the sum of three bf16 numbers of 8 each: the upper half (the largest numbers
// too), the upper half of what is left, and the rest.  Two parts, 16 bits, turned up to
// 0.3% of bf16 results into their neighbours, three 0.02%, for 94.5 us instead of 92.0 on
// the 4099 rows below; of rank 128 (4096 rows beside 59136 x 8192) 416 instead of 387.
//
// Launches: the first product (K split over workgroups, partial sums in the workspace)
// and the second one.  Up to 64 rows every workgroup of the first finds the rows of its
// adapter itself, one of them tells the second.  Beyond, a launch before them orders
// the rows by adapter into blocks of up to 64; with more than 512 a launch between them
// joins the splits, which otherwise every workgroup of the second sums for its rows.
// Ordering the whole call counts: blocks of 64 neighbouring rows each with its own
// adapters read A two and a half times on requests of 40 rows (246 us where 91 were then).
//
// What bounds it, measured (in a graph, beside 10240 x 8192 in three slices unless
// said): one token of rank 16 8.0 us, two launches of 4.2 and 4.9, each a chain of
// three round trips to memory; 16 requests of ranks to 64 beside 59136 x 8192 34.7 us, of
// which 28 the second launch, 83 MB (B's rows are lines of 128 bytes, however much of
// them an adapter's rank uses) by waves that wait for their one tile; 251 rows of which
// 166 have five of 64 adapters, 1032 -> 2561, 22 us, of which 13 the second launch, whose
// 88 workgroups are all on one XCD (see skinny_lora_expand); 4099 rows of rank
// 64, three adapters, 93.5 us = 6 + 35 + 6.5 + 49: the last adds to y at 3.4 TB/s, the
// first product waits for A (2.2 MB for every 64 rows, from the L2 cache).  4096 rows of
// rank 128 beside 59136 x 8192 426 us, of which some 355 the second launch, y at 2.7 TB/s
// beside three parts' matrix instructions; four tiles of ranks per wave of
// skinny_lora_shrink_many, which gate and up have there, spill 19 registers.
//   Tried with two parts of A x.  Whole lines: see Lines; 114 to 92 us on the 4099 rows.
// Odd rows of y by dwords: 26 to 21.5 us (251 rows).  Loads in branches of their own wait for
// each other; clamped addresses instead: 38 to 31 us (32 adapters of rank 128).  Tried
// and no faster: blocks of 128 rows (92 us; 30 for 24 on 1024 rows), two tiles of
// columns per wave (37.4 for 34.3 on the 16 requests), workgroups of 16 waves for few
// rows (9.1 for 8.5 on one token), K's stages in another order for every block.

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRowBlock = 64;          // rows of a block, all of one adapter
constexpr int kPiece = 64;             // values of K per row and wave at a time: a cache line
constexpr int kCols = 64;              // columns of y of a wave
constexpr int kMaxSlices = SKINNY_LORA_MAX_SLICES;

struct LoraArgs {
  const __bf16* x;
  const __bf16* base;
  __bf16* y;
  const int* ids;
  const int* ranks;
  const float* scale;
  // In the workspace:
  float* part;                         // [splits][slices][rows][rank]: A x over a split's K
  __bf16* low;                         // joined: [slices][rows][kParts][padded], A x in parts
  int4* blocks;                        // [most_blocks]: up to 64 rows of one adapter (-1: of
                                       // none): adapter, first place in order, rows, its rank
  int* order;                          // row numbers
  int most_blocks;
  int chunk_rows, chunk_blocks;        // many rows: those that are ordered together
  const __bf16* a[kMaxSlices];
  const __bf16* b[kMaxSlices];
  int n[kMaxSlices], col[kMaxSlices];  // columns of a slice, and the first one's number in y
  int tile[kMaxSlices + 1];            // first column tile of a slice
  int rows, adapters, rank, K, N, slices;
  int splits, pieces;                  // of K, and pieces of a split
  int rank_groups;                     // few rows: of 16 MT ranks; many: passes over A's tiles
  int ordinals;                        // few rows: adapters at most
  int copy;                            // base is not y: rows without an adapter are copied
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) {
  return __builtin_bit_cast(float, u & 0xffff0000u);
}

// 128 bytes of each of 16 rows in two registers' worth of 16 bytes per lane: as the
// products take them, lane (c, g) has parts g and g + 4 of row c; as they are loaded
// and stored, part l % 8 of rows l / 8 and l / 8 + 8, neighbouring lanes the parts of a
// row.  A load's cost in the L1 cache goes by the lines that each 16 neighbouring lanes
// touch: 16 rows apart an instruction of 1 KB takes some 66 cycles of a CU, 256 bytes in
// a row some 23.  The wave turns one form into the other in a buffer of its own; its
// accesses to shared memory are done in order.
constexpr int kTurn = 128;             // 16-byte parts of the buffer
__device__ __forceinline__ int line_row() { return (threadIdx.x & 63) >> 3; }
__device__ __forceinline__ int line_part() { return threadIdx.x & 7; }
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
struct Lines {
  u32x4 x[2];
  // Two rows fill the banks once: parts are turned by the number of their pair.
  static __device__ __forceinline__ int place(int row, int part) {
    return row * 8 + (part ^ (row >> 1));
  }
  __device__ __forceinline__ void to_products(u32x4* buf) {
    const int c = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    in_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) buf[place(line_row() + 8 * h, line_part())] = x[h];
    in_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) x[h] = buf[place(c, g + 4 * h)];
  }
  __device__ __forceinline__ void to_lines(u32x4* buf) {
    const int c = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    in_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) buf[place(c, g + 4 * h)] = x[h];
    in_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) x[h] = buf[place(line_row() + 8 * h, line_part())];
  }
};
// The same of 64 bytes of each of 16 rows, which a lane has one part of: l % 4 of row
// l / 4, or g of row c.
__device__ __forceinline__ void narrow_to_products(u32x4& x, u32x4* buf) {
  const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
  in_order();
  buf[l / 4 * 4 + ((l % 4) ^ (l >> 4))] = x;
  in_order();
  x = buf[c * 4 + (g ^ (c >> 2))];
}

__device__ __forceinline__ unsigned upper_halves(float a, float b) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, b), __builtin_bit_cast(unsigned, a),
                               0x07060302u);
}
// x - part; 0 for infinities, which part has in full.
__device__ __forceinline__ float rest_of(float x, float part) {
  const float r = x - part;
  return r - r == 0.0f ? r : 0.0f;
}
// Two fp32 numbers as the sums of kParts bf16 numbers each, largest first.
constexpr int kParts = 3;
struct Parts {
  unsigned p[kParts];
  __device__ __forceinline__ Parts(float x, float y) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      p[i] = upper_halves(x, y);
      x = rest_of(x, bf16_lo(p[i]));
      y = rest_of(y, bf16_hi(p[i]));
    }
  }
};

// The numbers of `rows`, side by side, the last one again behind them (one wave).
__device__ __forceinline__ void list_rows(unsigned long long rows, int* list) {
  const int lane = threadIdx.x & 63;
  const int count = __popcll(rows);
  if (rows >> lane & 1) list[__popcll(rows & ((1ull << lane) - 1))] = lane;
  if (lane >= count && count) list[lane] = 63 - __builtin_clzll(rows);
}

// Few rows (one block): A x for RT tiles of 16 rows and MT tiles of 16 ranks over a
// split's share of K: the waves take pieces of K in turn, and their sums are added
// in order.
constexpr int kFewWaves = 8;
constexpr int kSumTiles = 4;           // tiles that the waves add up at a time
template <int MT, int RT>
__device__ __forceinline__ void shrink(const LoraArgs& a, const __bf16* w, int rank, int r0,
                                       int count, int split, int slice, const int* list,
                                       u32x4* turn, float* sums) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  f32x4 acc[MT * RT];
#pragma unroll
  for (int i = 0; i < MT * RT; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const int lr = line_row(), lp = 8 * line_part();
  const __bf16* xp[RT][2];
  const __bf16* wp[MT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int t = 0; t < RT; ++t) xp[t][h] = a.x + (size_t)list[16 * t + 8 * h + lr] * a.K + lp;
#pragma unroll
    for (int m = 0; m < MT; ++m)
      wp[m][h] = w + (size_t)min(r0 + 16 * m + 8 * h + lr, rank - 1) * a.K + lp;
  }
  const int end = min((split + 1) * a.pieces * kPiece, a.K);
  for (int k = (split * a.pieces + wave) * kPiece; k < end; k += kFewWaves * kPiece) {
    Lines xf[RT], wf[MT];
    const bool in = k + lp < end;
    const int at = in ? k : -lp;       // chunks behind K's end: the row's first, and zeros for it
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int m = 0; m < MT; ++m) wf[m].x[h] = *reinterpret_cast<const u32x4*>(wp[m][h] + at);
#pragma unroll
      for (int t = 0; t < RT; ++t) xf[t].x[h] = *reinterpret_cast<const u32x4*>(xp[t][h] + at);
    }
    if (k + kPiece > end) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < MT; ++m) wf[m].x[h] = in ? wf[m].x[h] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < RT; ++t) xf[t].x[h] = in ? xf[t].x[h] : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) wf[m].to_products(turn);
#pragma unroll
    for (int t = 0; t < RT; ++t) xf[t].to_products(turn);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[m * RT + t] = mfma_bf16(wf[m].x[h], xf[t].x[h], acc[m * RT + t]);
  }
  // Lane (c, g), register r of a tile holds rank 4g + r of row c.
#pragma unroll
  for (int i0 = 0; i0 < MT * RT; i0 += kSumTiles) {
#pragma unroll
    for (int i = i0; i < i0 + kSumTiles && i < MT * RT; ++i)
      *reinterpret_cast<f32x4*>(sums + (wave * kSumTiles + i - i0) * 256 + lane * 4) = acc[i];
    __syncthreads();
    const int i = i0 + (int)threadIdx.x / 64;
    if (i < i0 + kSumTiles && i < MT * RT) {
      const int row = i % RT * 16 + c, r = r0 + 16 * (i / RT) + 4 * g;
      f32x4 s{0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kFewWaves; ++v)
        s += *reinterpret_cast<const f32x4*>(sums + (v * kSumTiles + i - i0) * 256 + lane * 4);
      if (row < count && r < rank)
        *reinterpret_cast<f32x4*>(
            a.part + ((size_t)(split * a.slices + slice) * a.rows + list[row]) * a.rank + r) = s;
    }
    __syncthreads();
  }
}

template <int MT>
__global__ __launch_bounds__(64 * kFewWaves) void skinny_lora_shrink_few(const LoraArgs a) {
  __shared__ int list[kRowBlock];
  __shared__ __attribute__((aligned(16))) float sums[kFewWaves * kSumTiles * 256];
  __shared__ __attribute__((aligned(16))) u32x4 turns[kFewWaves][kTurn];
  u32x4* turn = turns[threadIdx.x >> 6];
  int i = blockIdx.x;
  const int split = i % a.splits;
  i /= a.splits;
  const int r0 = i % a.rank_groups * 16 * MT;
  i /= a.rank_groups;
  const int slice = i % a.slices;
  const int ordinal = i / a.slices;
  // Lane l has row l's adapter; the workgroup takes the ordinal-th one that comes.
  const int lane = threadIdx.x & 63;
  int id = lane < a.rows ? a.ids[lane] : -1;
  if (id < 0 || id >= a.adapters) id = -1;
  unsigned long long rest = __ballot(id >= 0), rows = 0;
  int adapter = -1;
  for (int d = 0; d <= ordinal && rest; ++d) {
    adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    rows = __ballot(id == adapter);
    rest &= ~rows;
    if (d < ordinal) rows = 0;
  }
  const int count = __popcll(rows);
  const int rank = count == 0 ? 0 : a.ranks ? min(max(uniform(a.ranks[adapter]), 0), a.rank) : a.rank;
  // What the second launch has to know; the last block has the rows without an adapter.
  const bool tells = split == 0 && slice == 0 && r0 == 0;
  if (threadIdx.x < 64) {
    list_rows(rows, list);
    in_order();
    if (tells) {
      if (lane < count) a.order[ordinal * kRowBlock + lane] = list[lane];
      if (lane == 0) a.blocks[ordinal] = int4{adapter, ordinal * kRowBlock, count, rank};
      if (ordinal == 0) {
        const unsigned long long none = __ballot(id < 0 && lane < a.rows);
        const int last = a.most_blocks - 1;
        if (none >> lane & 1)
          a.order[last * kRowBlock + __popcll(none & ((1ull << lane) - 1))] = lane;
        if (lane == 0) a.blocks[last] = int4{-1, last * kRowBlock, __popcll(none), 0};
      }
    }
  }
  if (!a.a[slice] || r0 >= rank) return;
  __syncthreads();
  const __bf16* w = a.a[slice] + (size_t)adapter * a.rank * a.K;
  if (count <= 16) {
    shrink<MT, 1>(a, w, rank, r0, count, split, slice, list, turn, sums);
  } else {
    constexpr int H = MT > 2 ? 2 : MT;               // registers for two tiles of ranks by 64 rows
#pragma unroll
    for (int m = 0; m < MT; m += H)
      if (r0 + 16 * m < rank)
        shrink<H, 4>(a, w, rank, r0 + 16 * m, count, split, slice, list, turn, sums);
  }
}

// Many rows: A x for all slices and ranks of RT tiles of 16 rows.  The rows of x pass
// through shared memory, a stage of 128 values of K ahead in registers, and each wave
// multiplies them with MT tiles of 16 ranks of its own, whose rows of A it loads
// itself, a stage ahead.
constexpr int kStage = 128;            // values of K
constexpr int kChunks = kStage / 8;    // 16-byte chunks of a row's stage
template <int MT, int RT>
__device__ __forceinline__ void shrink_rows(const LoraArgs& a, int adapter, int rank, int count,
                                            int split, int pass, const int* list, u32x4* xs,
                                            u32x4* turn) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int per = (a.rank + 15) / 16;                // tiles of a slice
  // The wave's tiles: of which slice (-1: none), their first rank, and where a lane's
  // part of their rows lies.
  const unsigned char* wp[MT];
  unsigned off[MT][2];
  int slice[MT], r0[MT];
  bool any = false;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    int tile = (pass * MT + m) * kWaves + wave;
    slice[m] = -1;
    r0[m] = 0;
    wp[m] = (const unsigned char*)a.x;               // nothing to read: any row will do
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s) {
      if (s >= a.slices || !a.a[s]) continue;
      if (tile >= 0 && tile < per && 16 * tile < rank) {
        slice[m] = s;
        r0[m] = 16 * tile;
        wp[m] = (const unsigned char*)(a.a[s] + (size_t)adapter * a.rank * a.K);
      }
      tile -= per;
    }
    any = any || slice[m] >= 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)        // below 2^31: an adapter's A has 2^30 values at most
      off[m][h] = ((slice[m] < 0 ? 0u : (unsigned)min(r0[m] + 8 * h + line_row(), rank - 1) * (unsigned)a.K) +
                   8 * line_part()) * 2;
  }
  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
  // Thread i moves chunk i % 16 of rows i / 16 + 16 t; a row's chunks lie turned by the
  // row's number, so that 16 rows' equal chunks are in different banks.
  const int row = threadIdx.x / kChunks, chunk = threadIdx.x % kChunks;
  const __bf16* xp[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) xp[t] = a.x + (size_t)list[16 * t + row] * a.K + 8 * chunk;
  const int begin = split * a.pieces * kPiece, end = min(begin + a.pieces * kPiece, a.K);
  u32x4 xr[RT];
  Lines wf[2][MT], wn[2][MT];
  // K's last stage may go on behind K's end: loads there are of K's last chunk, and
  // count as zeros when they are used.
  const auto load_x = [&](int k) {
    const int d = min(k, a.K - 8 - 8 * chunk);
#pragma unroll
    for (int t = 0; t < RT; ++t) xr[t] = *reinterpret_cast<const u32x4*>(xp[t] + d);
  };
  const auto load_w = [&](int k) {
    unsigned d[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) d[u] = 2 * min(k + 64 * u, a.K - 8 - 8 * line_part());
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wn[u][m].x[h] = *reinterpret_cast<const u32x4*>(wp[m] + (off[m][h] + d[u]));
  };
  load_x(begin);
  load_w(begin);
  int buf = 0;
  for (int k = begin; k < end; k += kStage) {
    u32x4* x = xs + buf * kRowBlock * kChunks;
    buf ^= 1;
    if (k + kStage > end) {
#pragma unroll
      for (int t = 0; t < RT; ++t) xr[t] = k + 8 * chunk < end ? xr[t] : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            wn[u][m].x[h] = k + 64 * u + 8 * line_part() < end ? wn[u][m].x[h] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) x[(16 * t + row) * kChunks + (chunk ^ row)] = xr[t];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        wf[u][m] = wn[u][m];
        wf[u][m].to_products(turn);
      }
    __syncthreads();
    if (k + kStage < end) {
      load_x(k + kStage);
      load_w(k + kStage);
    }
    if (any) {
      // The next 32 values' rows of x come while these are multiplied.
      u32x4 xf[2][RT];
      const auto read = [&](int u) {
#pragma unroll
        for (int t = 0; t < RT; ++t) xf[u % 2][t] = x[(16 * t + c) * kChunks + ((4 * u + g) ^ c)];
      };
      read(0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u < 3) read(u + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][t] = mfma_bf16(wf[u / 2][m].x[u % 2], xf[u % 2][t], acc[m][t]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = r0[m] + 4 * g;
    if (slice[m] < 0 || r >= rank) continue;
#pragma unroll
    for (int t = 0; t < RT; ++t)
      if (16 * t + c < count)
        *reinterpret_cast<f32x4*>(a.part + ((size_t)(split * a.slices + slice[m]) * a.rows +
                                            list[16 * t + c]) * a.rank + r) = acc[m][t];
  }
  __syncthreads();
}

// The block that a workgroup works on.
struct Block {
  int adapter, first, count, rank;
  __device__ __forceinline__ Block(const LoraArgs& a, int i) {
    const int4 b = a.blocks[i];
    adapter = uniform(b.x);
    first = uniform(b.y);
    count = uniform(b.z);
    rank = uniform(b.w);
  }
  // Its rows' numbers, the last one again behind them.
  __device__ __forceinline__ void rows(const LoraArgs& a, int* list) const {
    if (threadIdx.x < kRowBlock) list[threadIdx.x] = a.order[first + min((int)threadIdx.x, count - 1)];
  }
};

template <int MT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void skinny_lora_shrink_many(const LoraArgs a) {
  __shared__ int list[kRowBlock];
  __shared__ __attribute__((aligned(16))) u32x4 xs[2 * kRowBlock * kChunks];
  __shared__ __attribute__((aligned(16))) u32x4 turns[kWaves][kTurn];
  u32x4* turn = turns[threadIdx.x >> 6];
  int i = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  if (i >= a.most_blocks * a.rank_groups * a.splits) return;
  const int block = i % a.most_blocks;
  i /= a.most_blocks;
  const int pass = i % a.rank_groups, split = i / a.rank_groups;
  const Block b(a, block);
  if (b.count == 0 || b.rank == 0) return;
  b.rows(a, list);
  __syncthreads();
  if (b.count <= 16) shrink_rows<MT, 1>(a, b.adapter, b.rank, b.count, split, pass, list, xs, turn);
  else shrink_rows<MT, 4>(a, b.adapter, b.rank, b.count, split, pass, list, xs, turn);
}

// Many rows: their order by adapter, and the blocks of up to 64 that share one (the
// blocks behind the last have no rows).  A workgroup counts its chunk of the rows in
// shared memory; in what order the rows of one adapter come changes no result.
constexpr int kGroupThreads = 1024;
__global__ __launch_bounds__(kGroupThreads) void skinny_lora_group(const LoraArgs a) {
  extern __shared__ int count[];                     // [adapters + 1], the last: without one
  __shared__ int2 waves[kGroupThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kinds = a.adapters + 1;
  const int row0 = blockIdx.x * a.chunk_rows, rows = min(a.rows - row0, a.chunk_rows);
  const int block0 = blockIdx.x * a.chunk_blocks;
  const int* ids = a.ids + row0;
  int* order = a.order + row0;
  int4* blocks = a.blocks + block0;
  for (int e = tid; e < kinds; e += kGroupThreads) count[e] = 0;
  __syncthreads();
  const auto kind_of = [&](int t) {
    const int e = ids[t];
    return e >= 0 && e < a.adapters ? e : a.adapters;
  };
  // The place of the row among its kind's: one addition for a wave of one kind.
  const auto place = [&](int e, bool live) -> int {
    const int first = uniform(e);
    const unsigned long long all = __ballot(live), same = __ballot(live && e == first);
    if (all == same) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&count[first], __popcll(all));
      return uniform(at) + __popcll(all & ((1ull << lane) - 1));
    }
    return live ? atomicAdd(&count[e], 1) : 0;
  };
  // Rows go by kBatch times the threads, whose kinds are loaded at once.  The first
  // batch's kinds and places stay in registers, the others' are found twice.
  constexpr int kBatch = 8;
  const auto load_kinds = [&](int t0, int (&kind)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) kind[i] = kind_of(min(t0 + i * kGroupThreads, rows - 1));
  };
  const auto place_all = [&](int t0, const int (&kind)[kBatch], int (&at)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = t0 + i * kGroupThreads;
      at[i] = t - lane < rows ? place(kind[i], t < rows) : 0;
    }
  };
  int kind[kBatch], at[kBatch];
  load_kinds(tid, kind);
  place_all(tid, kind, at);
  __syncthreads();                     // the first batch's come first among their kind
  for (int t0 = tid + kBatch * kGroupThreads; t0 - lane < rows; t0 += kBatch * kGroupThreads) {
    int k[kBatch], p[kBatch];
    load_kinds(t0, k);
    place_all(t0, k, p);
  }
  __syncthreads();
  // Rows and blocks of the kinds before each one's.
  const int per = (kinds + kGroupThreads - 1) / kGroupThreads;
  const int e0 = min(tid * per, kinds), e1 = min(e0 + per, kinds);
  int2 own{0, 0};
  for (int e = e0; e < e1; ++e) {
    own.x += count[e];
    own.y += (count[e] + kRowBlock - 1) / kRowBlock;
  }
  int2 incl = own;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const int x = __shfl_up(incl.x, off), y = __shfl_up(incl.y, off);
    if (lane >= off) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 63) waves[wave] = incl;
  __syncthreads();
  int2 before{incl.x - own.x, incl.y - own.y};
  int used = 0;
  for (int w = 0; w < kGroupThreads / 64; ++w) {
    if (w < wave) {
      before.x += waves[w].x;
      before.y += waves[w].y;
    }
    used += waves[w].y;
  }
  for (int e = e0; e < e1; ++e) {
    const int n = count[e];
    if (n == 0) continue;
    count[e] = before.x;                             // now the place of its first row
    const bool one = e < a.adapters;
    const int rank = !one ? 0 : a.ranks ? min(max(a.ranks[e], 0), a.rank) : a.rank;
    for (int r = 0; r < n; r += kRowBlock)
      blocks[before.y++] = int4{one ? e : -1, row0 + before.x + r, min(n - r, kRowBlock), rank};
    before.x += n;
  }
  for (int b = used + tid; b < a.chunk_blocks; b += kGroupThreads) blocks[b] = int4{-1, 0, 0, 0};
  __syncthreads();
  const auto write_all = [&](int t0, const int (&place)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t0 + i * kGroupThreads < rows) order[place[i]] = row0 + t0 + i * kGroupThreads;
  };
#pragma unroll
  for (int i = 0; i < kBatch; ++i) at[i] += count[kind[i]];
  write_all(tid, at);
  if (rows <= kBatch * kGroupThreads) return;
  __syncthreads();
  place_all(tid, kind, at);            // each kind's counter moves on by them
  __syncthreads();
  for (int t0 = tid + kBatch * kGroupThreads; t0 - lane < rows; t0 += kBatch * kGroupThreads) {
    load_kinds(t0, kind);
    place_all(t0, kind, at);
    write_all(t0, at);
  }
}

// Many rows: the splits' sums, times the scale, in the bf16 numbers that the products
// with B take; zeros behind the adapter's rank.
__global__ __launch_bounds__(kThreads) void skinny_lora_join(const LoraArgs a, int padded) {
  const int quads = padded / 4;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int r = (int)(i % quads) * 4;
  const long long at = i / quads;                    // slice * rows + row
  if (at >= (long long)a.slices * a.rows) return;
  const int slice = (int)(at / a.rows), row = (int)(at - (long long)slice * a.rows);
  const int e = a.ids[row];
  bool bare = true;
#pragma unroll
  for (int s = 0; s < kMaxSlices; ++s)
    if (s == slice) bare = !a.a[s];
  if (e < 0 || e >= a.adapters || bare) return;
  const int rank = a.ranks ? min(max(a.ranks[e], 0), a.rank) : a.rank;
  const float scale = a.scale ? a.scale[e] : 1.0f;
  const size_t step = (size_t)a.slices * a.rows * a.rank;
  const float* src = a.part + (size_t)at * a.rank + r;
  f32x4 s{0, 0, 0, 0};
  if (r < rank)
#pragma unroll 8
    for (int k = 0; k < a.splits; ++k) s += *reinterpret_cast<const f32x4*>(src + k * step);
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = r + e < rank ? s[e] * scale : 0.0f;
  const Parts v(s[0], s[1]), w(s[2], s[3]);
  __bf16* dst = a.low + (size_t)at * kParts * padded + r;
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    *reinterpret_cast<u32x2*>(dst + i * padded) = u32x2{v.p[i], w.p[i]};
}

// The columns of B that one wave multiplies: product j's row i is column 32 (j / 2) +
// 8 (i / 4) + 4 (j % 2) + i % 4, so that a lane ends with two runs of 8 neighbouring
// columns of one row of y, 32 apart, and four lanes with 32 neighbouring ones.
template <int KS>
struct Columns {
  u32x4 w[KS][4];
  static __device__ __forceinline__ int column(int j, int i, int n0, int n) {
    return min(n0 + 32 * (j >> 1) + 8 * (i >> 2) + 4 * (j & 1) + (i & 3), n - 1);
  }
  __device__ __forceinline__ void load(const __bf16* b, int pool, int rank, int n0, int n) {
    // Lanes past the adapter's rank read its first part again, for cut to drop: loads
    // in branches of their own would wait for each other.
    const auto at = [&](int r) { return r < rank ? r : 0; };
    if constexpr (KS == 1) {           // rows of up to 64 bytes, side by side
      const int l = threadIdx.x & 63, r = at(8 * (l & 3));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[0][j] = *reinterpret_cast<const u32x4*>(b + (size_t)column(j, l >> 2, n0, n) * pool + r);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __bf16* row = b + (size_t)column(j, 8 * h + line_row(), n0, n) * pool;
#pragma unroll
          for (int k = 0; k < KS; k += 2)
            w[k + h][j] = *reinterpret_cast<const u32x4*>(row + at(32 * k + 8 * line_part()));
        }
    }
  }
  // As the products take them.
  __device__ __forceinline__ void to_products(u32x4* buf) {
    if constexpr (KS == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) narrow_to_products(w[0][j], buf);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          Lines l = Lines{{w[k][j], w[k + 1][j]}};
          l.to_products(buf);
          w[k][j] = l.x[0];
          w[k + 1][j] = l.x[1];
        }
    }
  }
  // Columns past the adapter's own rank count as 0, whatever they hold.
  __device__ __forceinline__ void cut(int rank) {
    if (rank == 32 * KS) return;
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 32 * k + 8 * g + 2 * e;
          if (r >= rank) w[k][j][e] = 0;
          else if (r + 1 >= rank) w[k][j][e] &= 0xffffu;
        }
  }
};

// A x of some of a block's rows, summed over the splits in order, times the scale, in its
// bf16 parts: row t's at dwords t * stride of each part's `most` rows, zeros behind the rank.
constexpr int kMaxSplits = 8;
// Rows that are staged at a time.  All 64 of ranks above 64 leave room for a workgroup less
// on a CU: of rank 128, 16 rows beside 59136 x 8192 62.2 us for 57.6, 4096 rows 484 for 416;
// of rank 256, 4096 rows beside 10240 x 8192, 374 for 298.
constexpr int staged_rows(int ks) { return ks <= 2 ? kRowBlock : kRowBlock / 2; }
__device__ __forceinline__ void stage(const LoraArgs& a, int slice, int rank, int padded, int count,
                                      const int* list, float scale, f32x4* sums, unsigned* staged,
                                      int most, int stride) {
  const int quads = padded / 4, items = count * quads;
  const size_t step = (size_t)a.slices * a.rows * a.rank;
  const auto put = [&](int row, int r, f32x4 s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = r + e < rank ? s[e] * scale : 0.0f;
    const Parts v(s[0], s[1]), w(s[2], s[3]);
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      *reinterpret_cast<u32x2*>(staged + (i * most + row) * stride + r / 2) = u32x2{v.p[i], w.p[i]};
  };
  const auto source = [&](int item, int& row, int& r) {
    row = item / quads;
    r = (item - row * quads) * 4;
    return a.part + ((size_t)slice * a.rows + list[row]) * a.rank + min(r, a.rank - 4);
  };
  if (items > kThreads / kMaxSplits) {
    for (int i = threadIdx.x; i < items; i += kThreads) {
      int row, r;
      const float* src = source(i, row, r);
      f32x4 s = *reinterpret_cast<const f32x4*>(src);
#pragma unroll
      for (int k = 1; k < kMaxSplits; ++k)
        if (k < a.splits) s += *reinterpret_cast<const f32x4*>(src + k * step);
      put(row, r, s);
    }
    return;
  }
  // Few items: a thread for each split.
  constexpr int lanes = kThreads / kMaxSplits;
  const int k = threadIdx.x / lanes, i = threadIdx.x % lanes;
  int row = 0, r = 0;
  f32x4 s{0, 0, 0, 0};
  if (i < items && k < a.splits)
    s = *reinterpret_cast<const f32x4*>(source(i, row, r) + k * step);
  sums[threadIdx.x] = s;
  __syncthreads();
  if (i < items && k == 0) {
#pragma unroll
    for (int j = 1; j < kMaxSplits; ++j) s += sums[j * lanes + threadIdx.x];
    put(row, r, s);
  }
}

// The same of rows that were joined before.
__device__ __forceinline__ void stage_joined(const LoraArgs& a, int slice, int padded, int count,
                                             const int* list, unsigned* staged, int most,
                                             int stride) {
  const int chunks = padded / 8;       // of 16 bytes, of a row's part
  for (int i = threadIdx.x; i < count * kParts * chunks; i += kThreads) {
    const int row = i / (kParts * chunks), at = i - row * kParts * chunks;
    const u32x4 v = *reinterpret_cast<const u32x4*>(
        a.low + ((size_t)slice * a.rows + list[row]) * kParts * padded + 8 * at);
    *reinterpret_cast<u32x4*>(staged + (at / chunks * most + row) * stride + at % chunks * 4) = v;
  }
}

// 16 rows' part of base or y, a wave's 64 columns, in whole lines: a lane has 8
// neighbouring columns, `left` of them in the slice, of two rows.
struct Tile {
  size_t at[2];
  Lines l;
};
__device__ __forceinline__ Tile load_base(const LoraArgs& a, const int* list, int t, int count,
                                          int column, int left) {
  Tile b;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    b.at[h] = (size_t)list[min(t + 8 * h + line_row(), count - 1)] * a.N + column;
    const unsigned short* src = (const unsigned short*)a.base + b.at[h];
    b.l.x[h] = u32x4{0, 0, 0, 0};
    if (left >= 8) {
      // Off a dword's border an access takes twice as long: dwords around it instead,
      // where the neighbouring values are the tensor's own.
      if ((reinterpret_cast<uintptr_t>(src) & 2) && b.at[h] > 0 && b.at[h] + 8 < (size_t)a.rows * a.N) {
        const u32x4 lo = *reinterpret_cast<const u32x4_dword*>(src - 1);
        const unsigned hi = *reinterpret_cast<const unsigned*>(src + 7);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          b.l.x[h][e] = __builtin_amdgcn_alignbyte(e < 3 ? lo[e + 1] : hi, lo[e], 2);
      } else {
        b.l.x[h] = *reinterpret_cast<const u32x4_any*>(src);
      }
    } else if (left > 0) {             // the last ones again behind them
      unsigned v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = src[min(e, left - 1)];
#pragma unroll
      for (int e = 0; e < 4; ++e) b.l.x[h][e] = v[2 * e] | v[2 * e + 1] << 16;
    }
  }
  return b;
}
__device__ __forceinline__ void store_y(const LoraArgs& a, const Tile& b, int t, int count, int left) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (t + 8 * h + line_row() >= count) continue;
    if (left >= 8) {
      unsigned short* dst = (unsigned short*)a.y + b.at[h];
      if (reinterpret_cast<uintptr_t>(dst) & 2) {
        const u32x4 v = b.l.x[h];
        u32x3 m;
#pragma unroll
        for (int e = 0; e < 3; ++e) m[e] = __builtin_amdgcn_alignbyte(v[e + 1], v[e], 2);
        dst[0] = (unsigned short)v[0];
        *reinterpret_cast<u32x3_dword*>(dst + 1) = m;
        dst[7] = (unsigned short)(v[3] >> 16);
      } else {
        *reinterpret_cast<u32x4_any*>(dst) = b.l.x[h];
      }
    } else if (left > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left)
          ((unsigned short*)a.y)[b.at[h] + e] = (unsigned short)(b.l.x[h][e / 2] >> (16 * (e % 2)));
    }
  }
}

// The part of y that a workgroup writes: a wave's 64 columns of a slice from wave0 on,
// of which a lane has 8 from `column` of y on, with `left` left in the slice.
struct Part {
  int slice, n, wave0, column, left;
  __device__ __forceinline__ Part(const LoraArgs& a, int tile) {
    slice = 0;
    while (tile >= a.tile[slice + 1]) ++slice;
    n = a.n[slice];
    wave0 = ((tile - a.tile[slice]) * kWaves + uniform(threadIdx.x >> 6)) * kCols;
    column = a.col[slice] + wave0 + 8 * line_part();
    left = n - wave0 - 8 * line_part();
  }
};

// Sums of a lane's row that came out as no numbers, once more, by all of A x: an infinity
// in B times a part of A x that is 0, because A x has few bits, is NaN, where A x times it
// is infinite.
template <int KS>
__device__ __forceinline__ void sum_again(const LoraArgs& a, f32x4 (&acc)[4], const __bf16* w, int rank,
                                          int n0, int n, const unsigned* staged, int row, int stride) {
  int g = (threadIdx.x & 63) >> 4;
  asm volatile("" : "+v"(g), "+v"(row));             // or addresses take registers in every turn
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s = acc[j][i];
      if (s == s) continue;
      const __bf16* b = w + (size_t)Columns<KS>::column(j, 4 * g + i, n0, n) * a.rank;
      s = 0.0f;
      for (int r = 0; r < rank && s == s; ++r) {
        float v = 0.0f;
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p)        // smallest first: every sum is exact
          v += (float)((const __bf16*)(staged + (p * staged_rows(KS) + row) * stride))[r];
        s = fmaf((float)b[r], v, s);
      }
      acc[j][i] = s;
    }
}

// y of a block's rows from t0 up to t1 in the wave's columns, 16 rows at a time; what
// the next 16 are added to comes while the products run.
template <int KS>
__device__ __forceinline__ void expand(const LoraArgs& a, const Columns<KS>& b, const __bf16* w,
                                       int rank, const Part& p, int t0, int t1, int count,
                                       const int* list, Tile& next, const unsigned* staged, int stride,
                                       u32x4* turn) {
  const int c = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  for (int t = t0; t < t1; t += 16) {
    Tile here = next;
    if (t + 16 < count) next = load_base(a, list, t + 16, count, p.column, p.left);
    f32x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(staged + (i * staged_rows(KS) + t - t0 + c) * stride +
                                                        16 * k + 4 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = mfma_bf16(b.w[k][j], v, acc[j]);
      }
    float all = 0.0f;                  // NaN if one of them is
#pragma unroll
    for (int j = 0; j < 4; ++j) all += (acc[j][0] + acc[j][1]) + (acc[j][2] + acc[j][3]);
    if (__builtin_expect(all != all && t + c < t1, 0))
      sum_again<KS>(a, acc, w, rank, p.wave0, p.n, staged, t - t0 + c, stride);
    here.l.to_products(turn);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned y = here.l.x[h][e];
        here.l.x[h][e] = pack_bf16(bf16_lo(y) + acc[2 * h + e / 2][2 * (e % 2)],
                                   bf16_hi(y) + acc[2 * h + e / 2][2 * (e % 2) + 1]);
      }
    here.l.to_lines(turn);
    store_y(a, here, t, count, p.left);
  }
}

// Rows without an adapter, in the wave's columns.
__device__ __forceinline__ void copy_rows(const LoraArgs& a, int column, int left, int count,
                                          const int* list) {
#pragma unroll 4
  for (int t = 0; t < count; t += 16)
    store_y(a, load_base(a, list, t, count, column, left), t, count, left);
}

// JOINED: A x's parts were made before; else every workgroup sums the splits of
// its rows here.
template <int KS, bool JOINED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(KS <= 2 ? 4 : KS == 4 ? 2 : 1)))
void skinny_lora_expand(const LoraArgs a) {
  __shared__ int list[kRowBlock];
  __shared__ __attribute__((aligned(16))) u32x4 turns[kWaves][kTurn];
  extern __shared__ __attribute__((aligned(16))) unsigned staged[];    // A x in its parts
  constexpr int padded = 32 * KS;
  constexpr int stride = padded / 2 + 4;             // dwords of a row, kept off the same banks
  u32x4* turn = turns[threadIdx.x >> 6];
  // Workgroups go to the eight XCDs in turn; each XCD takes a run of neighbouring
  // parts of the same rows.  The blocks that have rows come first, before those that the
  // pool's adapters might have had: a call of few of a large pool's adapters works on few
  // of the XCDs.
  const int i = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  const int tiles = a.tile[a.slices];
  const int block = i / tiles;
  if (block >= a.most_blocks) return;
  const Block bl(a, block);
  if (bl.count == 0) return;
  const Part p(a, i - block * tiles);
  bl.rows(a, list);
  if (bl.rank == 0 || !a.a[p.slice]) {
    __syncthreads();
    if (a.copy && p.wave0 < p.n) copy_rows(a, p.column, p.left, bl.count, list);
    return;
  }
  Columns<KS> b;
  const __bf16* w = a.b[p.slice] + (size_t)bl.adapter * p.n * a.rank;
  b.load(w, a.rank, bl.rank, p.wave0, p.n);
  const float scale = !JOINED && a.scale ? a.scale[bl.adapter] : 1.0f;
  __syncthreads();
  Tile next = load_base(a, list, 0, bl.count, p.column, p.left);
  constexpr int most = staged_rows(KS);
  for (int t0 = 0; t0 == 0 || (most < kRowBlock && t0 < bl.count); t0 += most) {
    const int t1 = min(t0 + most, bl.count);
    if (t0) __syncthreads();           // the rows before these are done
    if constexpr (JOINED) stage_joined(a, p.slice, padded, t1 - t0, list + t0, staged, most, stride);
    else stage(a, p.slice, bl.rank, padded, t1 - t0, list + t0, scale, (f32x4*)turns, staged, most, stride);
    __syncthreads();
    if (p.wave0 >= p.n) continue;
    if (t0 == 0) {
      b.to_products(turn);
      b.cut(bl.rank);
    }
    expand<KS>(a, b, w, bl.rank, p, t0, t1, bl.count, list, next, staged, stride, turn);
  }
}

// ---------------------------------------------------------------------------
// Host side.

// How a call is cut: from the sizes alone, so that the workspace is known.
struct Cut {
  bool few;                            // one row block, no launch to group the rows
  bool join;                           // A x is joined by a launch of its own
  int tiles;                           // of 16 ranks in a workgroup (few) or a wave (many)
  int groups;                          // of them
  int splits, pieces, ordinals, most_blocks;
  int chunks, chunk_rows, chunk_blocks;
};
// Workgroups of the first product to cut a call into, if it is long enough.  128 to 512 of
// few rows are within 4% of each other, 1024 takes 19.6 us for 18.2 (16 rows of rank 64) and
// 34.2 for 31.7 (beside 59136 x 8192); 256 of many rows take 103 us for 92 (4096 of rank 64)
// and 454 for 425 (rank 128, 59136 x 8192), 1024 what 512 do.
constexpr int kFewGroups = 256;
constexpr int kManyGroups = 512;
constexpr int kChunkRows = 4096;
// Up to here every workgroup of the second launch sums its rows' splits itself.  A launch
// that joins them takes 24.4 us for 21.8 on 251 odd rows of rank 32 and 26.1 for 25.9 on 300
// of rank 16, 37.4 for 39.9 on 512 of rank 64, 63.5 for 70.9 on 2000.  Where y is wide and
// ranks are large it gains below, too: 126 for 177 on 512 rows of rank 128 beside 59136 x 8192.
constexpr int kJoinRows = 512;
Cut cut_of(const skinny_lora& l, int rows) {
  Cut c{};
  const int blocks = (rows + kRowBlock - 1) / kRowBlock;
  const int per = (l.rank + 15) / 16;                // rank tiles of a slice
  const int pieces = (l.K + kPiece - 1) / kPiece;
  const int most = rows < l.adapters ? rows : l.adapters;
  c.few = blocks == 1;
  long long splits;
  if (c.few) {
    c.ordinals = most < kRowBlock ? most : kRowBlock;
    c.most_blocks = c.ordinals + 1;                  // the last one: rows without an adapter
    splits = (pieces + kFewWaves - 1) / kFewWaves;   // one piece per wave
    if (splits > kMaxSplits) splits = kMaxSplits;
    c.tiles = per >= 4 ? 4 : per >= 2 ? 2 : 1;
    while (c.tiles > 1 && c.ordinals * l.slices * splits * ((per + c.tiles - 1) / c.tiles) < kFewGroups)
      c.tiles /= 2;
    c.groups = (per + c.tiles - 1) / c.tiles;
  } else {
    c.join = rows > kJoinRows;
    // Rows are ordered in chunks of some kChunkRows (one for 4096 rows takes 7 us, for
    // 16384 23), fewer where there are so many adapters that parts of blocks, of which
    // every chunk may have one for each kind of rows, would outnumber full blocks.
    c.chunks = (rows + kChunkRows - 1) / kChunkRows;
    if (c.chunks > blocks / (l.adapters + 1)) c.chunks = blocks / (l.adapters + 1);
    if (c.chunks < 1) c.chunks = 1;
    c.chunk_rows = (rows + c.chunks - 1) / c.chunks;
    c.chunks = (rows + c.chunk_rows - 1) / c.chunk_rows;
    const int kinds = c.chunk_rows < l.adapters + 1 ? c.chunk_rows : l.adapters + 1;
    c.chunk_blocks = (c.chunk_rows + kRowBlock - 1) / kRowBlock + kinds;
    if (c.chunk_blocks > c.chunk_rows) c.chunk_blocks = c.chunk_rows;
    c.most_blocks = c.chunks * c.chunk_blocks;
    int slices = 0;
    for (int i = 0; i < l.slices; ++i) slices += l.a[i] != nullptr;
    const int waves = (slices * per + kWaves - 1) / kWaves;        // tiles per wave
    c.groups = (waves + 3) / 4;
    c.tiles = (waves + c.groups - 1) / c.groups;
    splits = kManyGroups / ((long long)blocks * c.groups);
    const int whole = (pieces + 7) / 8;              // four stages
    if (splits > whole) splits = whole;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < 1) splits = 1;
  }
  c.pieces = (int)((pieces + splits - 1) / splits);
  if (!c.few) c.pieces = (c.pieces + 1) / 2 * 2;     // whole stages
  c.splits = (pieces + c.pieces - 1) / c.pieces;
  return c;
}

int padded_rank(const skinny_lora& l) {
  return l.rank <= 32 ? 32 : l.rank <= 64 ? 64 : l.rank <= 128 ? 128 : 256;
}

skinny_status check_lora(const skinny_lora* l, int rows, long long* width) {
  if (!l || rows < 1) return SKINNY_ERR_INVALID_ARG;
  if (l->adapters < 1 || l->rank < 1 || l->K < 1 || l->slices < 1) return SKINNY_ERR_INVALID_ARG;
  if (l->slices > SKINNY_LORA_MAX_SLICES) return SKINNY_ERR_UNSUPPORTED;
  long long n = 0;
  bool any = false;
  for (int i = 0; i < l->slices; ++i) {
    if (l->n[i] < 1 || (l->a[i] != nullptr) != (l->b[i] != nullptr)) return SKINNY_ERR_INVALID_ARG;
    if (!aligned(l->a[i], 16) || !aligned(l->b[i], 16)) return SKINNY_ERR_UNSUPPORTED;
    n += l->n[i];
    any = any || l->a[i];
  }
  if (!any) return SKINNY_ERR_INVALID_ARG;
  if (rows > SKINNY_LORA_MAX_ROWS || l->adapters > SKINNY_LORA_MAX_ADAPTERS || l->rank % 8 != 0 ||
      l->rank > SKINNY_LORA_MAX_RANK || l->K % 8 != 0 || (long long)l->K * l->rank > (1 << 30) || n > (1 << 28))
    return SKINNY_ERR_UNSUPPORTED;
  if (!aligned(l->ranks, 4) || !aligned(l->scale, 4)) return SKINNY_ERR_UNSUPPORTED;
  *width = n;
  return SKINNY_OK;
}

// The workspace's parts, each 16-byte aligned.
struct Space {
  size_t low, blocks, order, bytes;
  Space(const skinny_lora& l, const Cut& c, int rows) {
    const size_t all = (size_t)l.slices * rows;
    low = c.splits * all * l.rank * sizeof(float);
    blocks = low + (c.join ? all * kParts * padded_rank(l) * sizeof(__bf16) : 0);
    order = blocks + (size_t)c.most_blocks * sizeof(int4);
    bytes = order + (c.few ? (size_t)c.most_blocks * kRowBlock : (size_t)rows) * sizeof(int);
    if (bytes < SKINNY_MIN_WORKSPACE_BYTES) bytes = SKINNY_MIN_WORKSPACE_BYTES;
  }
};

size_t workspace_of(const skinny_lora& l, int rows) { return Space(l, cut_of(l, rows), rows).bytes; }

template <int KS, bool JOINED>
skinny_status launch_expand(const LoraArgs& a, unsigned grid, hipStream_t stream) {
  constexpr int lds = kParts * staged_rows(KS) * (16 * KS + 4) * (int)sizeof(unsigned);
  constexpr int rest = kRowBlock * (int)sizeof(int) + kWaves * kTurn * (int)sizeof(u32x4);
  static_assert(lds + rest <= 64 * 1024, "more shared memory than a launch may have unasked");
  hipLaunchKernelGGL((skinny_lora_expand<KS, JOINED>), dim3(grid), dim3(kThreads), lds, stream, a);
  return hipGetLastError() == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP;
}
template <bool JOINED>
skinny_status launch_expand(const LoraArgs& a, int padded, unsigned grid, hipStream_t stream) {
  if (padded == 32) return launch_expand<1, JOINED>(a, grid, stream);
  if (padded == 64) return launch_expand<2, JOINED>(a, grid, stream);
  if (padded == 128) return launch_expand<4, JOINED>(a, grid, stream);
  return launch_expand<8, JOINED>(a, grid, stream);
}

}  // namespace

extern "C" {

size_t skinny_lora_workspace_bytes(const skinny_lora* lora, int rows) {
  long long n;
  return check_lora(lora, rows, &n) == SKINNY_OK ? workspace_of(*lora, rows) : 0;
}

skinny_status skinny_lora_linear(const skinny_lora* lora, const void* x, const int* ids, int rows,
                                 const void* base, void* y, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  long long width = 0;
  skinny_status st = check_lora(lora, rows, &width);
  if (st != SKINNY_OK) return st;
  const skinny_lora& l = *lora;
  if (!x || !ids || !y) return SKINNY_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(y, 2) || !aligned(base, 2))
    return SKINNY_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < workspace_of(l, rows)) return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_UNSUPPORTED;
  if (!base) base = y;
  const size_t yb = (size_t)rows * width * 2;
  const Range yr = range_of(y, yb), wr = range_of(workspace, workspace_bytes);
  Range in[5 + 2 * SKINNY_LORA_MAX_SLICES];
  int m = 0;
  in[m++] = range_of(x, (size_t)rows * l.K * 2);
  in[m++] = range_of(ids, (size_t)rows * 4);
  if (l.ranks) in[m++] = range_of(l.ranks, (size_t)l.adapters * 4);
  if (l.scale) in[m++] = range_of(l.scale, (size_t)l.adapters * 4);
  for (int i = 0; i < l.slices; ++i) {
    if (!l.a[i]) continue;
    in[m++] = range_of(l.a[i], (size_t)l.adapters * l.rank * l.K * 2);
    in[m++] = range_of(l.b[i], (size_t)l.adapters * l.rank * l.n[i] * 2);
  }
  if (base != y) in[m++] = range_of(base, yb);
  if (overlap(yr, wr)) return SKINNY_ERR_INVALID_ARG;
  for (int i = 0; i < m; ++i)
    if (overlap(yr, in[i]) || overlap(wr, in[i])) return SKINNY_ERR_INVALID_ARG;

  const Cut c = cut_of(l, rows);
  LoraArgs a;
  a.x = (const __bf16*)x;
  a.base = (const __bf16*)base;
  a.y = (__bf16*)y;
  a.ids = ids;
  a.ranks = l.ranks;
  a.scale = l.scale;
  a.part = (float*)workspace;
  a.rows = rows;
  a.adapters = l.adapters;
  a.rank = l.rank;
  a.K = l.K;
  a.N = (int)width;
  a.slices = l.slices;
  a.splits = c.splits;
  a.pieces = c.pieces;
  const Space space(l, c, rows);
  a.low = (__bf16*)((char*)workspace + space.low);
  a.order = (int*)((char*)workspace + space.order);
  a.blocks = (int4*)((char*)workspace + space.blocks);
  a.most_blocks = c.most_blocks;
  a.chunk_rows = c.chunk_rows;
  a.chunk_blocks = c.chunk_blocks;
  a.rank_groups = c.groups;
  a.ordinals = c.ordinals;
  a.copy = base != y;
  int col = 0, tile = 0;
  for (int i = 0; i < kMaxSlices; ++i) {
    const bool in_use = i < l.slices;
    a.a[i] = in_use ? (const __bf16*)l.a[i] : nullptr;
    a.b[i] = in_use ? (const __bf16*)l.b[i] : nullptr;
    a.n[i] = in_use ? l.n[i] : 0;
    a.col[i] = col;
    a.tile[i] = tile;
    col += a.n[i];
    tile += (a.n[i] + kCols * kWaves - 1) / (kCols * kWaves);
  }
  a.tile[kMaxSlices] = tile;
  for (int i = l.slices; i < kMaxSlices; ++i) a.tile[i] = tile;
  const long long first = c.few ? (long long)a.ordinals * a.slices * a.rank_groups * a.splits
                                : ((long long)c.most_blocks * a.rank_groups * a.splits + 7) / 8 * 8;
  const long long second = ((long long)c.most_blocks * tile + 7) / 8 * 8;
  const int padded = padded_rank(l);
  const long long join = ((long long)l.slices * rows * (padded / 4) + kThreads - 1) / kThreads;
  if (first * (c.few ? 64 * kFewWaves : kThreads) > 0xffffffffLL ||      // threads of a launch
      second * kThreads > 0xffffffffLL || join * kThreads > 0xffffffffLL)
    return SKINNY_ERR_UNSUPPORTED;
  DeviceInfo d;
  st = device_info(&d);
  if (st != SKINNY_OK) return st;
  if (!d.gfx950) return SKINNY_ERR_UNSUPPORTED;

  const hipStream_t hs = (hipStream_t)stream;
  const dim3 grid((unsigned)first), few(64 * kFewWaves), many(kThreads);
  if (c.few) {
    if (c.tiles == 1) hipLaunchKernelGGL(skinny_lora_shrink_few<1>, grid, few, 0, hs, a);
    else if (c.tiles == 2) hipLaunchKernelGGL(skinny_lora_shrink_few<2>, grid, few, 0, hs, a);
    else hipLaunchKernelGGL(skinny_lora_shrink_few<4>, grid, few, 0, hs, a);
  } else {
    hipLaunchKernelGGL(skinny_lora_group, dim3(c.chunks), dim3(kGroupThreads),
                       (size_t)(l.adapters + 1) * sizeof(int), hs, a);
    if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
    if (c.tiles == 1) hipLaunchKernelGGL(skinny_lora_shrink_many<1>, grid, many, 0, hs, a);
    else if (c.tiles == 2) hipLaunchKernelGGL(skinny_lora_shrink_many<2>, grid, many, 0, hs, a);
    else if (c.tiles == 3) hipLaunchKernelGGL(skinny_lora_shrink_many<3>, grid, many, 0, hs, a);
    else hipLaunchKernelGGL(skinny_lora_shrink_many<4>, grid, many, 0, hs, a);
    if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
    if (c.join) hipLaunchKernelGGL(skinny_lora_join, dim3((unsigned)join), many, 0, hs, a, padded);
  }
  if (hipGetLastError() != hipSuccess) return SKINNY_ERR_HIP;
  return c.join ? launch_expand<true>(a, padded, (unsigned)second, hs)
                : launch_expand<false>(a, padded, (unsigned)second, hs);
}

}  // extern "C"
