// Microscaled 4-bit floating point (MXFP4): quantisation, its inverse, and products on
// tcgen05.mma.kind::mxf4 for sm_100a.
//
// Format: 32 consecutive values along K share a scale 2^X, X = floor(log2 max|v|) - 2 clamped to
// [-127, 127] (-127 for a zero block), stored as the UE8M0 byte X + 127; a value is the E2M1 code of
// v 2^-X (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign bit; nearest, ties to the even code, saturating at
// 6), two codes to a byte, the first in the low half.  A block that holds a NaN or an infinity has
// no such scale: its byte is 255 (UE8M0's NaN), and it stands for NaNs.
//
// Elements are row-major, cols / 2 bytes a row.  Scales are stored as the tensor core reads them:
// the scales of 128 rows and 128 columns (4 blocks) form a 512-byte atom, byte 16 i + 4 j + b = row
// i + 32 j, block b (i < 32, j < 4, b < 4), which one tcgen05.cp copies into four TMEM columns.
// Atoms are stored row tile by row tile, two per 256 columns (one k-block of the products).  Blocks
// past the last column have scale byte 0: their elements read as zeros, and 0 times a finite scale
// adds nothing.  Rows come in groups (one for a plain matrix, an expert's rows, an expert's weight
// matrix), and every group's atoms start with a tile of their own, so a tile of 128 rows never mixes
// the scales of two groups, wherever the groups begin in the elements.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"

namespace lmoe {

constexpr int kMx4MaxGroups = 1024;

__host__ __device__ __forceinline__ int mx4_kblocks(int cols) { return (cols + 255) / 256; }

// How the rows of a matrix fall into groups.
struct Mx4Rows {
  const int* offsets;  // device, [groups + 1]: first row of each group and the end; null: equal groups
  int groups;
  int rows;            // of the whole matrix
};

// Tiles of 128 rows, group by group.  Ragged groups need a prefix sum over the groups, which each
// block makes once in shared memory.
struct Mx4Tiles {
  const int* first_row;      // shared, [groups + 1] (ragged groups)
  const uint16_t* partial;   // shared, [groups + 1]: partial tiles, see first_tile
  int groups, group_rows, tiles_per_group, total;
  int rest_lo, rest_hi;   // rows [0, rest_lo) and [rest_hi, rows) belong to no group

  // First tile of group g: the whole tiles that its distance from the first row would make, and what
  // rounding each group up to whole tiles adds to them, which is at most one a group (16 bits).
  __device__ __forceinline__ int first_tile(int g) const { return ((first_row[g] - first_row[0]) >> 7) + partial[g]; }
  // Group, first row and valid rows of tile t; the whole warp takes part (two rounds of 32 groups
  // compared at once).
  __device__ __forceinline__ void get(int t, int& g, int& row0, int& valid) const {
    if (first_row) {
      // the last group whose first tile is at most t (groups without rows begin where the next one does)
      const int lane = threadIdx.x & 31;
      const int step = (groups + 31) >> 5;
      const int a = lane * step;
      const int base = (__popc(__ballot_sync(0xffffffffu, a < groups && first_tile(a) <= t)) - 1) * step;
      const int b = base + lane;
      g = base + __popc(__ballot_sync(0xffffffffu, lane < step && b < groups && first_tile(b) <= t)) - 1;
      const int within = (t - first_tile(g)) * 128;
      row0 = first_row[g] + within;
      valid = min(128, first_row[g + 1] - row0);
    } else {
      g = t / tiles_per_group;
      const int within = (t - g * tiles_per_group) * 128;
      row0 = g * group_rows + within;
      valid = min(128, group_rows - within);
    }
  }
};

constexpr int kMx4TableInts = (kMx4MaxGroups + 1) + (kMx4MaxGroups + 2) / 2 + 1 + 8;

// Fills the tile table (at least 256 threads, every thread of the block takes part; ends with a
// barrier).  Offsets that
// decrease or leave [0, rows] are recorded as LMOE_STATUS_BAD_INDEX and give no tiles at all, so no
// access follows from them (every row then belongs to no group).
__device__ inline Mx4Tiles mx4_tiles(const Mx4Rows& r, int* table, uint32_t* status) {
  Mx4Tiles t;
  t.groups = r.groups;
  if (!r.offsets) {
    t.first_row = nullptr;
    t.partial = nullptr;
    t.group_rows = r.rows / r.groups;
    t.tiles_per_group = (t.group_rows + 127) >> 7;
    t.total = t.tiles_per_group * r.groups;
    t.rest_lo = 0;
    t.rest_hi = r.rows;
    return t;
  }
  int* first_row = table;
  uint16_t* partial = reinterpret_cast<uint16_t*>(table + kMx4MaxGroups + 1);
  int* bad = table + (kMx4MaxGroups + 1) + (kMx4MaxGroups + 2) / 2;
  int* wsum = bad + 1;
  const int n = r.groups, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) *bad = 0;
  __syncthreads();
  // the first 256 threads take four groups each (kMx4MaxGroups in all)
  int sum = 0, own[4] = {0, 0, 0, 0};
  if (tid < 256) {
    int v[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = r.offsets[min(tid * 4 + j, n)];
    bool wrong = false;
#pragma unroll
    for (int j = 0; j < 5; ++j) wrong |= v[j] < 0 || v[j] > r.rows || (j && v[j] < v[j - 1]);
    if (wrong) *bad = 1;
#pragma unroll
    for (int j = 0; j < 5; ++j)
      if (tid * 4 + j <= n && (j < 4 || tid == 255)) first_row[tid * 4 + j] = v[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      own[j] = wrong ? 0 : (v[j + 1] - v[j] + 127) >> 7;  // 0 past the last group
      sum += own[j];
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    sum = inc - sum;  // before this thread's groups, within the warp
  }
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) sum += wsum[w];
    base += wsum[w];
  }
  if (tid < 256) {
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int g = tid * 4 + j;
      if (g <= n && (j < 4 || tid == 255)) partial[g] = (uint16_t)(sum - ((first_row[g] - first_row[0]) >> 7));
      if (j < 4) sum += own[j];
    }
  }
  __syncthreads();
  t.first_row = first_row;
  t.partial = partial;
  t.group_rows = t.tiles_per_group = 0;
  t.total = *bad ? 0 : base;
  t.rest_lo = *bad ? r.rows : first_row[0];
  t.rest_hi = *bad ? r.rows : first_row[n];
  if (*bad && tid == 0) set_status(status, LMOE_STATUS_BAD_INDEX);
  return t;
}

// Zeroes row i of the rows that belong to no group, for i = first, first + stride, ... (a warp a row).
template <typename T>
__device__ __forceinline__ void mx4_zero_rest(const Mx4Tiles& t, int rows, T* out, long long ld, int cols, int first,
                                              int stride, int lane) {
  const int n = t.rest_lo + rows - t.rest_hi;
  for (int i = first; i < n; i += stride) {
    T* row = out + (long long)(i < t.rest_lo ? i : t.rest_hi + i - t.rest_lo) * ld;
    for (int c = lane; c < cols; c += 32) row[c] = from_f<T>(0.f);
  }
}

// --------------------------------------------------------------------------- quantisation
// Scale byte of a block whose largest magnitude has the fp32 bits `amax` (NaN and infinity compare
// above every number): the exponent field less 2, so that the largest value lands in [4, 8).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// Eight values, scaled, as eight codes (the first in the lowest four bits).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float s) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[2 * j] * s, v[2 * j + 1] * s), __NV_E2M1, cudaRoundNearest)
         << (8 * j);
  return w;
}

// Eight values of a row as they are stored (bf16: four words, fp32: eight); `vec`: the row starts on a
// 16-byte boundary.
template <typename T>
struct Mx4Raw {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void mx4_load8(const T* p, bool vec, Mx4Raw<T>& r) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 q = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = q.x;
      r.w[4 * i + 1] = q.y;
      r.w[4 * i + 2] = q.z;
      r.w[4 * i + 3] = q.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = (uint32_t)h[2 * j] | ((uint32_t)h[2 * j + 1] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = reinterpret_cast<const uint32_t*>(p)[j];
  }
}
// Largest magnitude of the eight values, as fp32 bits (for bf16 the low half may hold anything: only the
// exponent is read).
__device__ __forceinline__ uint32_t mx4_amax(const Mx4Raw<bf16>& r) {
  const uint32_t m = __vmaxu2(__vmaxu2(r.w[0] & 0x7FFF7FFFu, r.w[1] & 0x7FFF7FFFu),
                              __vmaxu2(r.w[2] & 0x7FFF7FFFu, r.w[3] & 0x7FFF7FFFu));
  return max(m, m << 16);
}
__device__ __forceinline__ uint32_t mx4_amax(const Mx4Raw<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, r.w[j] & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ void mx4_floats(const Mx4Raw<bf16>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(r.w[j] << 16);
    v[2 * j + 1] = __uint_as_float(r.w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void mx4_floats(const Mx4Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j]);
}

struct Mx4QuantParams {
  const void* src;   // [rows, ld]; PAIRED: w1 [groups, h, cols]
  const void* src3;  // PAIRED: w3
  long long ld;
  int cols;
  Mx4Rows rows;
  uint8_t* elems;
  uint8_t* scales;
  uint32_t* status;
  int vec;           // every row of src starts on a 16-byte boundary
};

// Row n (0 .. 15) of slice `sl` (0 .. 7) of a tile: a slice's rows are those whose scale words lie side by
// side in an atom (bytes 64 sl .. +63).
__device__ __forceinline__ int mx4_slice_row(int sl, int n) { return 4 * sl + (n >> 2) + 32 * (n & 3); }

// A warp takes a slice of 16 rows and 256 columns of a tile at a time; a lane holds 8 of a row's
// values, four lanes a block of 32, so a warp reads a row's 256 values at once and writes their codes
// as one 128-byte line.  Of the scale byte that a block's four lanes agree on, lane j keeps that of rows
// 4 q + j; two exchanges of bytes between lanes then give each lane the four bytes of one row (half-warp
// a: atom a, lane n of it: row n), which leave as two runs of 64 bytes.  No shared memory and no
// barriers but for the ragged groups' table: the warps' loads overlap freely.
// PAIRED: rows are the gate and linear projections of a SwiGLU interleaved in groups of 64 (row
// 128 (j / 64) + j % 64 = w1[j], 64 further w3[j]).
constexpr int kMx4Batch = 4;  // rows in flight a warp
template <typename T, bool PAIRED>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 4) mx4_quant_kernel(const Mx4QuantParams p) {
  __shared__ int table[kMx4TableInts];
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, table, p.status);
  const int lane = threadIdx.x & 31;
  const unsigned nkb = (unsigned)mx4_kblocks(p.cols);
  const unsigned n = (unsigned)tiles.total * nkb * 8;  // less than 2^31, as the host has seen to
  for (unsigned u = blockIdx.x * 8 + (threadIdx.x >> 5); u < n; u += gridDim.x * 8) {
    const int sl = (int)(u & 7);
    const unsigned tk = u >> 3;
    const int t = (int)(tk / nkb), kb = (int)(tk - t * nkb);
    int g, row0, valid;
    tiles.get(t, g, row0, valid);
    const int c = kb * 256 + lane * 8;
    const bool in = c < p.cols;  // cols is a multiple of 32: a block is inside or outside whole
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 16; b += kMx4Batch) {
      Mx4Raw<T> raw[kMx4Batch];
#pragma unroll
      for (int i = 0; i < kMx4Batch; ++i) {
        const int r = mx4_slice_row(sl, b + i);
#pragma unroll
        for (int j = 0; j < (int)(2 * sizeof(T)); ++j) raw[i].w[j] = 0;
        if (in && r < valid) {
          const int row = row0 + r;
          if constexpr (PAIRED) {
            // row of the interleaved matrix -> row of w1 or w3 (group g has 2h rows)
            const int within = row - g * tiles.group_rows;
            const long long srow = (long long)g * (tiles.group_rows >> 1) + (within >> 7) * 64 + (within & 63);
            mx4_load8(static_cast<const T*>((within & 64) ? p.src3 : p.src) + srow * p.ld + c, p.vec, raw[i]);
          } else {
            mx4_load8(static_cast<const T*>(p.src) + (long long)row * p.ld + c, p.vec, raw[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kMx4Batch; ++i) {
        const int r = mx4_slice_row(sl, b + i);
        uint32_t amax = mx4_amax(raw[i]);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const uint32_t sb = mx4_scale_byte(amax);
        // 2^-X = 2^(127 - byte): exponent field 254 - byte, at least 2 for every finite block
        const float s = __uint_as_float((254u - min(sb, 252u)) << 23);
        if (in && r < valid) {
          float v[8];
          mx4_floats(raw[i], v);
          *reinterpret_cast<uint32_t*>(p.elems + (long long)(row0 + r) * (p.cols >> 1) + (c >> 1)) = e2m1x8(v, s);
        }
        if ((lane & 3) == ((b + i) & 3)) word |= sb << (8 * ((b + i) >> 2));
      }
    }
    // bytes (block (lane >> 2) & 3, q = 0 .. 3) -> (row 4 ((lane >> 2) & 3) + lane % 4, block = 0 .. 3)
    uint32_t y = __shfl_xor_sync(0xffffffffu, word, 4);
    word = __byte_perm(word, y, (lane & 4) ? 0x3715 : 0x6240);
    y = __shfl_xor_sync(0xffffffffu, word, 8);
    word = __byte_perm(word, y, (lane & 8) ? 0x3276 : 0x5410);
    // row n of the slice: byte 16 (4 sl + n / 4) + 4 (n % 4) = 64 sl + 4 n of its atom
    *reinterpret_cast<uint32_t*>(p.scales + (size_t)tk * 1024 + (lane >> 4) * 512 + 64 * sl + 4 * (lane & 15)) = word;
  }
}

// --------------------------------------------------------------------------- dequantisation
struct Mx4DequantParams {
  const uint8_t* elems;
  const uint8_t* scales;
  void* out;         // [rows, ld]
  long long ld;
  int cols;
  Mx4Rows rows;
  uint32_t* status;
  int vec;
  int zero_rest;     // 1: rows of no group are set to zero
};

// The values of eight codes (the first in the lowest four bits) times s; fp16 holds every code's value.
__device__ __forceinline__ void e2m1_values(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w >> (8 * j)), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x * s;
    v[2 * j + 1] = f.y * s;
  }
}

// Same slices and lanes as the quantisation.
template <typename T>
__global__ void __launch_bounds__(256, 5) mx4_dequant_kernel(const Mx4DequantParams p) {
  __shared__ int table[kMx4TableInts];
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, table, p.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned nkb = (unsigned)mx4_kblocks(p.cols);
  const unsigned n = (unsigned)tiles.total * nkb * 8;
  for (unsigned u = blockIdx.x * 8 + warp; u < n; u += gridDim.x * 8) {
    const int sl = (int)(u & 7);
    const unsigned tk = u >> 3;
    const int t = (int)(tk / nkb), kb = (int)(tk - t * nkb);
    int g, row0, valid;
    tiles.get(t, g, row0, valid);
    const int c = kb * 256 + lane * 8;
    const bool in = c < p.cols;
    const uint32_t word =
        *reinterpret_cast<const uint32_t*>(p.scales + (size_t)tk * 1024 + (lane >> 4) * 512 + 64 * sl + 4 * (lane & 15));
#pragma unroll 1
    for (int b = 0; b < 16; b += 8) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = mx4_slice_row(sl, b + i);
        w[i] = 0;
        if (in && r < valid)
          w[i] = *reinterpret_cast<const uint32_t*>(p.elems + (long long)(row0 + r) * (p.cols >> 1) + (c >> 1));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = mx4_slice_row(sl, b + i);
        const uint32_t sb = (__shfl_sync(0xffffffffu, word, (lane & 16) + b + i) >> (8 * ((lane >> 2) & 3))) & 255u;
        // 2^(byte - 127): a subnormal for byte 0, NaN for 255
        const float s = sb == 255u ? __uint_as_float(0x7FC00000u)
                                   : (sb ? __uint_as_float(sb << 23) : __uint_as_float(0x00400000u));
        float v[8];
        e2m1_values(w[i], s, v);
        if (!in || r >= valid) continue;
        T* o = static_cast<T*>(p.out) + (long long)(row0 + r) * p.ld + c;
        if (p.vec) {
          if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = from_f<T>(v[j]);
        }
      }
    }
  }
  if (p.zero_rest)
    mx4_zero_rest(tiles, p.rows.rows, static_cast<T*>(p.out), p.ld, p.cols, blockIdx.x * 8 + warp, gridDim.x * 8, lane);
}

}  // namespace lmoe
