// Products of MXFP4 matrices on the tensor cores: C[M, N] = A[M, K] B[N, K]^T, or, grouped, the rows
// of group g of A times matrix g of B.  tcgen05.mma.kind::mxf4 multiplies the 4-bit codes exactly,
// scales each 32-element block's products by its two operands' scales and accumulates in fp32.
//
// Tiles of 128 rows and 128 columns, k-blocks of 256 (128 bytes of codes: one swizzle row, four MMAs
// of K = 64, two scales of each row an MMA).  CTA = 10 warps: warp 0 loads a k-block's operand tiles
// (TMA) and scale atoms (bulk copies) into a ring, warp 1 copies the atoms into TMEM (two buffers by
// k-block parity) and issues the MMAs, warps 2-9 drain the other accumulator.
#pragma once

#include "mx4.cuh"

namespace lmoe {

struct Mx4GemmParams {
  CUtensorMap tmA;  // codes [M, K / 2] u8, box 128 x 128
  CUtensorMap tmB;  // codes [groups N, K / 2] u8, box 128 x 128
  const uint8_t* a_sf;
  const uint8_t* b_sf;
  Mx4Rows rows;     // A's groups
  int N;            // rows of each B matrix
  int n_tiles;      // ceil(N / 128)
  int nkb;          // k-blocks of 256
  void* c;          // [M, N], or [M, N / 2] for the SwiGLU form
  long long ldc;
  int c_cols;       // columns of c
  int zero_rest;    // 1: rows of c that belong to no group are set to zero
  int vec;          // every row of c starts on a 16-byte boundary
  uint32_t* status;
};

constexpr int kMx4Stages = 6;
constexpr int kMx4StageBytes = 2 * 16384 + 2 * 1024;
constexpr int kMx4BarOffset = kMx4Stages * kMx4StageBytes;
constexpr int kMx4TableOffset = kMx4BarOffset + 256;
constexpr int kMx4SmemBytes = kMx4TableOffset + 4 * kMx4TableInts + 1024;
constexpr int kMx4Threads = 320;
constexpr int kMx4EpiWarps = 8;

// Instruction descriptor, kind::mxf4: D fp32, A and B E2M1 (both K-major), UE8M0 scales, M = m,
// N = n, K = 64; sf (0 or 2) selects the half of each scale word the MMA reads.
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, int m, int sf) {
  return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 7) << 27) | ((uint32_t)sf << 29);
}
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}

// 32 consecutive values of a row of c, those before column `cols` only.
template <typename T>
__device__ __forceinline__ void mx4_store32(T* row, int c0, int cols, bool vec, const float (&v)[32]) {
  constexpr int W = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < 32; j += W) {
    if (vec && c0 + j + W <= cols) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(row + c0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      else
        *reinterpret_cast<uint4*>(row + c0 + j) =
            make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]), pack_bf16x2(v[j + 4], v[j + 5]),
                       pack_bf16x2(v[j + 6], v[j + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (c0 + j + i < cols) row[c0 + j + i] = from_f<T>(v[j + i]);
    }
  }
}

template <typename T, bool GLU>
__global__ void __launch_bounds__(kMx4Threads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4GemmParams p) {
  constexpr int S = kMx4Stages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kMx4BarOffset);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kMx4EpiWarps);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // TMEM columns: accumulators [0, 256); scales of k-block parity i at 256 + 64 i: A's two atoms at
  // +0 and +4, B's at +32 and +36
  const uint32_t sf_base = tmem_base + 256;
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, reinterpret_cast<int*>(smem + kMx4TableOffset), p.status);
  const long long num_tiles = (long long)tiles.total * p.n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- loads
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true;
      for (long long tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x) {
        const int mt = (int)(tile / p.n_tiles), nt = (int)(tile - (long long)mt * p.n_tiles);
        int g, row0, valid;
        tiles.get(mt, g, row0, valid);
        const int brow0 = g * p.N + nt * 128;
        const uint8_t* asf = p.a_sf + (size_t)mt * p.nkb * 1024;
        const uint8_t* bsf = p.b_sf + ((size_t)g * p.n_tiles + nt) * p.nkb * 1024;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort, p.status)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = smem + stage * kMx4StageBytes;
          mbar_expect_tx(&full[stage], kMx4StageBytes);
          tma_load_2d(a_dst, &p.tmA, &full[stage], kb * 128, row0);
          tma_load_2d(a_dst + 16384, &p.tmB, &full[stage], kb * 128, brow0);
          bulk_load(a_dst + 32768, asf + (size_t)kb * 1024, 1024, &full[stage]);
          bulk_load(a_dst + 32768 + 1024, bsf + (size_t)kb * 1024, 1024, &full[stage]);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok)
        for (int i = 0; i < S; ++i)
          if ((armed >> i) & 1u) mbar_drain(&full[i], (armed_parity >> i) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (long long tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x, ++it) {
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, abort, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 128;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * kMx4StageBytes);
          const uint32_t b_addr = a_addr + 16384;
          const uint32_t sfa = sf_base + (kb & 1) * 64, sfb = sfa + 32;
          tc_cp_atom(sfa, a_addr + 32768);
          tc_cp_atom(sfa + 4, a_addr + 32768 + 512);
          tc_cp_atom(sfb, a_addr + 32768 + 1024);
          tc_cp_atom(sfb + 4, a_addr + 32768 + 1536);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_mxf4(d_tmem, smem_desc_sw128(a_addr + k * 32), smem_desc_sw128(b_addr + k * 32),
                        idesc_mxf4(128, 128, 2 * (k & 1)), sfa + 4 * (k >> 1), sfb + 4 * (k >> 1), (kb | k) != 0);
          tc_commit(&empty[stage]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit(&tfull[acc]);
      }
      if (!ok) {
        tc_commit(drain);
        mbar_drain(drain, 0);
      }
    }
  } else {
    // ---------------- epilogue warps 2..9: TMEM lane quarter (warp % 4), column half (warp - 2) / 4
    const int wq = warp & 3;
    const int half_id = (warp - 2) >> 2;
    const int rl = wq * 32 + lane;
    int it = 0;
    bool ok = true;
    for (long long tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x, ++it) {
      const int mt = (int)(tile / p.n_tiles), nt = (int)(tile - (long long)mt * p.n_tiles);
      int g, row0, valid;
      tiles.get(mt, g, row0, valid);
      T* crow = static_cast<T*>(p.c) + (long long)(row0 + rl) * p.ldc;
      const int acc = it & 1;
      ok = mbar_wait(&tfull[acc], (it >> 1) & 1, abort, p.status);
      __syncwarp();
      if (__any_sync(0xffffffffu, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(wq * 32) << 16) + acc * 128;
      if constexpr (GLU) {
        // gate columns [32 half, +32), linear columns 64 further
        uint32_t gv[32], uv[32];
        tmem_ld32(tbase + half_id * 32, gv);
        tmem_ld32(tbase + 64 + half_id * 32, uv);
        tc_wait_ld();
        float a[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = silu_fast(__uint_as_float(gv[i])) * __uint_as_float(uv[i]);
        if (rl < valid) mx4_store32(crow, nt * 64 + half_id * 32, p.c_cols, p.vec, a);
      } else {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          uint32_t v[32];
          tmem_ld32(tbase + half_id * 64 + j * 32, v);
          tc_wait_ld();
          float a[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(v[i]);
          if (rl < valid) mx4_store32(crow, nt * 128 + half_id * 64 + j * 32, p.c_cols, p.vec, a);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
    if (p.zero_rest)
      mx4_zero_rest(tiles, p.rows.rows, static_cast<T*>(p.c), p.ldc, p.c_cols, blockIdx.x * kMx4EpiWarps + warp - 2,
                    gridDim.x * kMx4EpiWarps, lane);
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace lmoe
