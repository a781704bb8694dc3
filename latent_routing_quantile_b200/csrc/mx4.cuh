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
// i + 32 j, block b (i < 32, j < 4, b < 4): lane i of four TMEM columns, a word a lane and column.
// Atoms are stored row tile by row tile, two per 256 columns (one k-block of the products).  Blocks
// past the last column have scale byte 0: their elements read as zeros, and 0 times a finite scale
// adds nothing.  Rows come in groups (one for a plain matrix, an expert's rows, an expert's weight
// matrix), and every group's atoms start with a tile of their own, so a tile of 128 rows never mixes
// the scales of two groups, wherever the groups begin in the elements.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace lmoe {

constexpr int kMx4MaxGroups = 1024;

__host__ __device__ __forceinline__ int mx4_kblocks(int cols) { return cols / 256 + (cols % 256 != 0); }

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

// Fills the tile table (at least 256 threads; every thread of the block takes part; ends with a
// barrier).  Offsets that decrease or leave [0, rows] are recorded as LMOE_STATUS_BAD_INDEX and give no
// tiles at all, so no access follows from them (every row then belongs to no group).
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
// Eight values as eight codes (the first in the lowest four bits), to nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// How rows are read and written: 32 bytes at a time, 16, or element by element, by what every row's
// address is a multiple of (quantising 16384 x 7168 bf16: 45.6, 45.9 and 127 us).
enum Mx4Access : int { MX4_ELEMENTS = 0, MX4_16 = 1, MX4_32 = 2 };

// Sixteen values of a row as they are stored (bf16: eight words, fp32: sixteen).
template <typename T>
struct Mx4Raw {
  uint32_t w[4 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void mx4_load16(const T* p, int access, Mx4Raw<T>& r) {
  constexpr int kWords = 4 * sizeof(T);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
  if (access == MX4_32) {
#pragma unroll
    for (int i = 0; i < kWords; i += 8)
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3]), "=r"(r.w[i + 4]),
                     "=r"(r.w[i + 5]), "=r"(r.w[i + 6]), "=r"(r.w[i + 7])
                   : "l"(q + i));
  } else if (access == MX4_16) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = ldg_nc_v4(q + i);
      r.w[i] = v.x;
      r.w[i + 1] = v.y;
      r.w[i + 2] = v.z;
      r.w[i + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < kWords; ++j) r.w[j] = (uint32_t)h[2 * j] | ((uint32_t)h[2 * j + 1] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < kWords; ++j) r.w[j] = q[j];
  }
}
// Exponent field of the largest magnitude of a block: two lanes' sixteen values each (255: it holds a NaN
// or an infinity, which compare above every number as integers).
__device__ __forceinline__ uint32_t mx4_exponent(const Mx4Raw<bf16>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __vmaxu2(m, r.w[j] & 0x7FFF7FFFu);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m >> 23, (m >> 7) & 0xFFu);
}
__device__ __forceinline__ uint32_t mx4_exponent(const Mx4Raw<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max(m, r.w[j] & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return m >> 23;
}
// Codes of the sixteen values times 2^-X, whose exponent field is 256 - e (e: the block's, at least 2).
// bf16 values are scaled two at a time: exact, but for results far below the smallest code, which stay
// there.
__device__ __forceinline__ uint2 mx4_codes(const Mx4Raw<bf16>& r, uint32_t e) {
  const uint32_t s = ((256u - e) << 7) * 0x10001u;
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r.w[j]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&s));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&x);
    v[2 * j] = __uint_as_float(w << 16);
    v[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}
__device__ __forceinline__ uint2 mx4_codes(const Mx4Raw<float>& r, uint32_t e) {
  const float s = __uint_as_float((256u - e) << 23);
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r.w[j]) * s;
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

struct Mx4QuantParams {
  const void* src;   // [rows, ld]; PAIRED: w1 [groups, h, cols]; INDEXED: [src_rows, ld]
  const void* src3;  // PAIRED: w3
  const int* index;  // INDEXED: src's row of each row of the matrix
  int src_rows;      // INDEXED: rows of src
  long long ld;
  int cols;
  Mx4Rows rows;
  uint8_t* elems;
  uint8_t* scales;
  uint32_t* status;
  int access;        // Mx4Access of src
};

// A tile's rows fall into eight slices of 16: row n of slice sl is row 4 sl + n / 4 + 32 (n % 4), so that
// a slice's scale words lie side by side in an atom (bytes 64 sl .. +63).  A warp takes a slice and 256
// columns of a tile at a time, half a warp a row: a lane reads 16 of its values and writes their eight
// bytes of codes, two lanes make a block of 32.  Lanes of a half: bit 3 the atom a, bits 1-2 the block b
// in it, bit 0 the lane j of the block.
__device__ __forceinline__ constexpr int mx4_row(int n) { return (n >> 2) + 32 * (n & 3); }

// Of the scale byte that a block's two lanes agree on, lane j of half h keeps those of rows
// n = 4 q + 2 j + h (q = 0 .. 3); two exchanges of bytes between the lanes of b then give each lane the
// four blocks' bytes of one row, which leave as runs of 64 bytes.  No shared memory and no barriers but
// for the ragged groups' table.
// Bound by memory: 16384 x 7168 bf16 takes 45 us, 6.5 TB/s of values read and codes written.  With 8
// values a lane the instructions bound it (60 us): 16 halve the maxima's exchanges and the scales'
// arithmetic for each value.
// MX4_PAIRED: rows are the gate and linear projections of a SwiGLU interleaved in groups of 64 (row
// 128 (j / 64) + j % 64 = w1[j], 64 further w3[j]).  MX4_INDEXED: row r is src's row index[r]; an index
// outside src is reported and gives a row of zeros.
enum Mx4Source : int { MX4_PLAIN = 0, MX4_PAIRED = 1, MX4_INDEXED = 2 };
template <typename T, int SOURCE>
__global__ void __launch_bounds__(256, 4) mx4_quant_kernel(const Mx4QuantParams p) {
  __shared__ int table[kMx4TableInts];
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;  // rows in flight a half-warp
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, table, p.status);
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const unsigned nkb = (unsigned)mx4_kblocks(p.cols);
  const unsigned n = (unsigned)tiles.total * nkb * 8;  // less than 2^31, as the host has seen to
  const long long pitch = p.cols >> 1;
  constexpr bool PAIRED = SOURCE == MX4_PAIRED, INDEXED = SOURCE == MX4_INDEXED;
  const long long to3 = PAIRED ? static_cast<const T*>(p.src3) - static_cast<const T*>(p.src) : 0;
  for (unsigned u = blockIdx.x * 8 + (threadIdx.x >> 5); u < n; u += gridDim.x * 8) {
    const int sl = (int)(u & 7);
    const unsigned tk = u >> 3;
    const int t = (int)(tk / nkb), kb = (int)(tk - t * nkb);
    int g, row0, valid;
    tiles.get(t, g, row0, valid);
    const int c = kb * 256 + (lane & 15) * 16;
    // the slice's first row
    const T* src;
    if constexpr (PAIRED) {
      // interleaved row -> row of w1 or w3 (group g has 2h rows): row n of a slice is one of w3's for
      // n % 4 = 2, 3
      const int within = row0 - g * tiles.group_rows;
      src = static_cast<const T*>(p.src) + ((long long)g * (tiles.group_rows >> 1) + (within >> 1) + 4 * sl) * p.ld + c;
    } else if constexpr (INDEXED) {
      src = static_cast<const T*>(p.src) + c;
    } else {
      src = static_cast<const T*>(p.src) + (long long)(row0 + 4 * sl) * p.ld + c;
    }
    int from = 0;  // INDEXED: lane n holds src's row of row n, -1 for none
    if constexpr (INDEXED) {
      const int r = 4 * sl + mx4_row(lane & 15);
      if (r < valid) from = p.index[row0 + r];
      if ((unsigned)from >= (unsigned)p.src_rows) {
        from = -1;
        set_status(p.status, LMOE_STATUS_BAD_INDEX);
      }
    }
    uint8_t* dst = p.elems + (long long)(row0 + 4 * sl) * pitch + (c >> 1);
    // rows from the slice's first on that exist (cols is a multiple of 32: a block is inside or outside)
    const int left = c < p.cols ? valid - 4 * sl : 0;
    uint32_t word = 0;
    auto rows = [&](auto whole) {
#pragma unroll
      for (int b = 0; b < 8; b += kBatch) {
        Mx4Raw<T> raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = mx4_row(2 * (b + i)) + 32 * half;  // row 2 (b + i) + half of the slice
          long long at = PAIRED ? (long long)(r & 63) * p.ld + ((r & 64) ? to3 : 0) : (long long)r * p.ld;
          bool some = decltype(whole)::value || r < left;
          if constexpr (INDEXED) {
            const int f = __shfl_sync(0xffffffffu, from, 2 * (b + i) + half);
            at = (long long)f * p.ld;
            some = some && f >= 0;
          }
          if (some) {
            mx4_load16(src + at, p.access, raw[i]);
          } else {
#pragma unroll
            for (int j = 0; j < (int)(4 * sizeof(T)); ++j) raw[i].w[j] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int step = b + i, r = mx4_row(2 * step) + 32 * half;
          const uint32_t ex = mx4_exponent(raw[i]);
          // scale byte: the exponent field less 2, so that the largest value lands in [4, 8)
          const uint32_t e = max(ex, 2u), sb = ex == 255u ? 255u : e - 2;
          if (decltype(whole)::value || r < left) *reinterpret_cast<uint2*>(dst + r * pitch) = mx4_codes(raw[i], e);
          if ((lane & 1) == (step & 1)) word |= sb << (8 * (step >> 1));
        }
      }
    };
    if (__all_sync(0xffffffffu, left >= 100)) rows(std::true_type()); else rows(std::false_type());  // 99 = 3 + 96
    // bytes (b, q = 0 .. 3) -> (q = b, blocks 0 .. 3)
    uint32_t y = __shfl_xor_sync(0xffffffffu, word, 2);
    word = __byte_perm(word, y, (lane & 2) ? 0x3715 : 0x6240);
    y = __shfl_xor_sync(0xffffffffu, word, 4);
    word = __byte_perm(word, y, (lane & 4) ? 0x3276 : 0x5410);
    // row n = 4 b + 2 j + h: byte 64 sl + 4 n of atom a
    const int row16 = 4 * ((lane >> 1) & 3) + 2 * (lane & 1) + half;
    *reinterpret_cast<uint32_t*>(p.scales + (size_t)tk * 1024 + ((lane >> 3) & 1) * 512 + 64 * sl + 4 * row16) = word;
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
  int access;        // Mx4Access of out
  int zero_rest;     // 1: rows of no group are set to zero
};

// The values of eight codes (the first in the lowest four bits) times s; fp16 holds every code's value.
__device__ __forceinline__ void e2m1_values(uint32_t w, float s, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x * s;
    v[2 * j + 1] = f.y * s;
  }
}
// Sixteen values of a row.
template <typename T>
__device__ __forceinline__ void mx4_store16v(T* o, int access, const float (&v)[16]) {
  uint32_t w[4 * sizeof(T)];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  }
  if (access == MX4_32) {
#pragma unroll
    for (int i = 0; i < (int)(4 * sizeof(T)); i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t*>(o) + i),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                   "r"(w[i + 7])
                   : "memory");
  } else if (access == MX4_16) {
#pragma unroll
    for (int i = 0; i < (int)(4 * sizeof(T)); i += 4)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(o) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = from_f<T>(v[j]);
  }
}

// Same slices and lanes as the quantisation.  16384 x 7168 to bf16: 49 us, 6.1 TB/s.
template <typename T>
__global__ void __launch_bounds__(256, 4) mx4_dequant_kernel(const Mx4DequantParams p) {
  __shared__ int table[kMx4TableInts];
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, table, p.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4;
  const unsigned nkb = (unsigned)mx4_kblocks(p.cols);
  const unsigned n = (unsigned)tiles.total * nkb * 8;
  const long long pitch = p.cols >> 1;
  for (unsigned u = blockIdx.x * 8 + warp; u < n; u += gridDim.x * 8) {
    const int sl = (int)(u & 7);
    const unsigned tk = u >> 3;
    const int t = (int)(tk / nkb), kb = (int)(tk - t * nkb);
    int g, row0, valid;
    tiles.get(t, g, row0, valid);
    const int c = kb * 256 + (lane & 15) * 16;
    const uint8_t* src = p.elems + (long long)(row0 + 4 * sl) * pitch + (c >> 1);
    T* dst = static_cast<T*>(p.out) + (long long)(row0 + 4 * sl) * p.ld + c;
    const int left = c < p.cols ? valid - 4 * sl : 0;
    // lane 16 a + n: the four scale bytes of row n in atom a
    const uint32_t word =
        *reinterpret_cast<const uint32_t*>(p.scales + (size_t)tk * 1024 + (lane >> 4) * 512 + 64 * sl + 4 * (lane & 15));
    auto rows = [&](auto whole) {
#pragma unroll
      for (int b = 0; b < 8; b += 4) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = mx4_row(2 * (b + i)) + 32 * half;
          w[i] = decltype(whole)::value || r < left ? *reinterpret_cast<const uint2*>(src + r * pitch) : make_uint2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int step = b + i, r = mx4_row(2 * step) + 32 * half;
          const uint32_t sw = __shfl_sync(0xffffffffu, word, ((lane << 1) & 16) + 2 * step + half);
          const uint32_t sb = (sw >> (8 * ((lane >> 1) & 3))) & 255u;
          // 2^(byte - 127); the extra bit makes byte 0 the subnormal 2^-127 and byte 255 a NaN
          const float s = __uint_as_float((sb << 23) | (((sb + 1) & 0xFEu) ? 0u : 0x00400000u));
          if (!decltype(whole)::value && r >= left) continue;
          float v[16];
          e2m1_values(w[i].x, s, v);
          e2m1_values(w[i].y, s, v + 8);
          mx4_store16v(dst + r * p.ld, p.access, v);
        }
      }
    };
    if (__all_sync(0xffffffffu, left >= 100)) rows(std::true_type()); else rows(std::false_type());
  }
  if (p.zero_rest)
    mx4_zero_rest(tiles, p.rows.rows, static_cast<T*>(p.out), p.ld, p.cols, blockIdx.x * 8 + warp, gridDim.x * 8, lane);
}

}  // namespace lmoe
