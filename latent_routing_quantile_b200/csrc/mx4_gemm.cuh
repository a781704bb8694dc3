// Products of MXFP4 matrices on the tensor cores: C[M, N] = A[M, K] B[N, K]^T, or, grouped, the rows
// of group g of A times matrix g of B.  tcgen05.mma.kind::mxf4 multiplies the 4-bit codes exactly,
// scales each 32-element block's products by its two operands' scales and accumulates in fp32.
//
// K-blocks of 256 (128 bytes of codes: one swizzle row, four MMAs of K = 64, two scales of each row
// an MMA).  CTA = 14 warps: warp 0 loads a k-block's operand tiles and scale atoms (TMA) into a ring,
// warps 10-13 write the atoms into TMEM, warp 1 issues the MMAs, warps 2-9 drain the other
// accumulator.  Tiles (rows x columns of C):
//   128 x 128: with split > 1 a cluster of `split` CTAs shares a tile, each a range of the k-blocks, and
//              adds the parts up through distributed shared memory in a fixed order;
//   128 x 256: a quarter less operand traffic per output.
//
// 256-wide accumulators: two of them and the scales do not fit TMEM's 512 columns, so the two share
// 128 columns ([0, 256) and [128, 384)).  The epilogue warps of that half signal when they have read
// them (tovl), and the next tile's MMAs start on that signal.
//
// Scales go from shared memory to TMEM through registers (tcgen05.st), by warps that do nothing else.
// tcgen05.cp would do without them, but it runs in the MMAs' queue and one after the other with them:
// six copies a k-block of a 128 x 256 tile took 420 of its 930 cycles.  Every stage of the ring
// has TMEM columns of its own, so writing them is ordered after the MMAs that last read them by the
// ring itself (they released the stage before it was loaded again).
//
// Measured: 16384 x 8192 x 7168 with the SwiGLU epilogue 356 us, 5.4 PFLOP/s (the MMAs alone 290 us, the
// loads alone 275); sustained, at the power cap's clock, 424 us.  The tensor pipe is the busiest unit, 73% of
// the cycles (a k-block of a 128 x 256 tile takes 702 of them, its MMAs 512), L2 at 62%, the banks of
// shared memory at 33% for reads and 28% for writes.  The wide layer's gate and linear projections (262144
// rows over 896 experts, 1024 x 2048) 344 us: MMAs alone 220, a quarter of them for the rows that fill up an
// expert's last tile, loads alone 224; a quarter of its tokens and experts keeps the tensor pipe busy for
// 52% of the cycles and DRAM for 53%.
#pragma once

#include "mx4.cuh"

namespace lmoe {

struct Mx4GemmParams {
  CUtensorMap tmA;   // codes [M, K / 2] u8, box 128 bytes x 128 rows
  CUtensorMap tmA32; // the same, boxes of 32 rows (tiles of at most 32 rows)
  CUtensorMap tmB;   // codes [groups N, K / 2] u8, box 128 bytes x the tile's width
  CUtensorMap tmSA;  // scale atoms, see make_map_atoms: one row tile a box
  CUtensorMap tmSB;  // one or two (256-wide tiles) row tiles a box
  CUtensorMap tmC;   // c, boxes of a staging round (mx4_store_rows); used when align is 16
  Mx4Rows rows;      // A's groups
  int N;             // rows of each B matrix
  int b_tiles;       // row tiles of each B matrix: ceil(N / 128)
  int n_tiles;       // tiles of C along N
  int nkb;           // k-blocks of 256
  int split;         // CTAs a tile (128 x 128 tiles only)
  void* c;           // [M, N], or [M, N / 2] for the SwiGLU form
  long long ldc;
  int c_cols;        // columns of c
  int zero_rest;     // 1: rows of c that belong to no group are set to zero
  int align;         // every row of c starts on a boundary of 16, 8, 4 or 2 bytes
  uint32_t* status;
};

constexpr int kMx4Threads = 448;
constexpr int kMx4EpiWarps = 8;
constexpr int kMx4StgBytes = kMx4EpiWarps * 2048;  // a staging box an epilogue warp

template <int BN>
struct Mx4Cfg {
  static constexpr int kABytes = 16384, kBBytes = BN * 128;
  static constexpr int kSBBytes = BN * 8;
  static constexpr int kStageBytes = kABytes + kBBytes + 1024 + kSBBytes;
  static constexpr int kStages = BN == 128 ? 6 : 4;
  static constexpr int kStgOffset = kStages * kStageBytes;
  static constexpr int kBarOffset = kStgOffset + kMx4StgBytes;
  static constexpr int kTableOffset = kBarOffset + 8 * (4 * kStages + 6) + 16;
  static constexpr int kSmemBytes = kTableOffset + 4 * kMx4TableInts;
  // TMEM columns: accumulators at 0 and 128, then the scales of each stage (A's 8 columns, B's BN / 16)
  static constexpr int kAcc1 = 128, kSfCols = 128 + BN, kSfBuf = 8 + BN / 16;
  static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
  static_assert(kStageBytes % 1024 == 0, "tiles start on 1024-byte boundaries");
  static_assert(kSfCols + kStages * kSfBuf <= 512, "tensor memory");
};

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
// Writes four consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}
constexpr int kMx4PartPitch = 132;  // floats from row to row of a split tile's parts

// Writes a staging round to rows of c on a boundary of UNIT (4 or 2) words: a unit a lane, neighbouring
// lanes a row's neighbouring units, rows before `valid` and columns before `cols` only.  c: the round's
// first row and column.
template <int UNIT, int kRows, int kChunks, int kShift, typename T>
__device__ __forceinline__ void mx4_store_units(const uint8_t* box, T* c, long long ldc, int cols, int valid, int lane) {
  using V = std::conditional_t<UNIT == 4, uint4, uint2>;
  constexpr int kLanes = 4 * kChunks / UNIT;         // lanes a row
  constexpr int kPer = 4 * UNIT / (int)sizeof(T);    // columns a unit
  const int l = lane % kLanes, r0 = lane / kLanes, first = l * UNIT;
  c += r0 * ldc + kPer * l;
  const int left = cols - kPer * l;
  auto unit = [&](int rr) {
    const int chunk = (first >> 2) ^ ((rr >> kShift) & (kChunks - 1));
    return box + rr * 16 * kChunks + 16 * chunk + 4 * (first & 3);
  };
  T* dst = c;
#pragma unroll
  for (int i = 0; i < kRows * kLanes / 32; ++i, dst += 32 / kLanes * ldc) {
    const int rr = i * (32 / kLanes) + r0;
    const V v = *reinterpret_cast<const V*>(unit(rr));
    if (rr < valid && left >= kPer) *reinterpret_cast<V*>(dst) = v;
  }
  if (left > 0 && left < kPer) {  // the unit that the last column lies in
#pragma unroll 1
    for (int rr = r0; rr < min(valid, kRows); rr += 32 / kLanes, c += 32 / kLanes * ldc)
      for (int j = 0; j < left; ++j) c[j] = reinterpret_cast<const T*>(unit(rr))[j];
  }
}
// The same for rows on any boundary: a word a lane.  A bf16 row on an odd boundary takes the words that
// lie in it, each put together from two of the box, and its first and last value by themselves.
template <int kRows, int kChunks, typename T>
__device__ __forceinline__ void mx4_store_words(const uint8_t* box, T* c, long long ldc, int cols, int valid, int lane) {
  constexpr int kLanes = 4 * kChunks;  // lanes a row: 32, or 16 for two rows at once
  const int l = lane % kLanes, r0 = lane / kLanes;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(box);
  c += r0 * ldc;
#pragma unroll 8  // 16: registers spill
  for (int i = 0; i < 16; ++i, c += 32 / kLanes * ldc) {
    const uint32_t w = words[32 * i + (lane ^ ((i & (kChunks - 1)) << 2))];
    const bool row = i * (32 / kLanes) + r0 < valid;
    if constexpr (sizeof(T) == 4) {
      if (row && l < cols) c[l] = __uint_as_float(w);
    } else {
      const int odd = (int)((uintptr_t)c >> 1) & 1, e = 2 * l + odd, end = min(2 * kLanes, cols);
      const uint32_t z = __funnelshift_r(w, __shfl_down_sync(0xffffffffu, w, 1), 16 * odd);
      if (row && e + 1 < end) *reinterpret_cast<uint32_t*>(c + e) = z;
      if (row && e + 1 == end) c[e] = __ushort_as_bfloat16((unsigned short)z);
      if (row && odd && l == 0 && end > 0) c[0] = __ushort_as_bfloat16((unsigned short)w);
    }
  }
}
// Rows a staging round holds: the box's 2 KB in rows of kWords words.
__host__ __device__ constexpr int mx4_round_rows(int words) { return 2048 / (4 * words); }

// Writes kWords words (64 or 128 bytes) of each of a warp's 32 rows of c, rows from `row`: lane l holds
// row row + l's.  They go through the warp's 2 KB staging box (32 rows of 64 bytes, or twice 16 rows of
// 128; 16-byte chunks swizzled as the tensor map of c says), which a TMA store then writes while the
// warp goes on.  A round with rows past `valid` (they may be another group's) or columns past p.c_cols, or
// of a c whose rows are not 16-byte aligned, is written by the lanes instead: in units of 16 or 8 bytes if
// every row starts on such a boundary, else in words.  13620 x N x 1536 in us: into bf16 rows 6080 wide 65,
// 6076 (8 bytes) 71 (in words 104), 6078 (4) 104, 6077 (2) 107; into fp32 rows 86, 6078 (8) 105 (in words
// 153), 6077 (4) 153.  What bounds those is each warp's instructions, so the loops have few.  A SwiGLU's
// rounds (16 words) leave out the 8-byte units: with their code its kernel spills registers, and 135000
// aligned rows of 384 values in 512 groups take 97 us for 71.  col: first column; columns past p.c_cols are
// not written.
template <int kWords, typename T>
__device__ __forceinline__ void mx4_store_rows(const Mx4GemmParams& p, uint8_t* box, const uint32_t (&w)[kWords],
                                               int row, int col, int valid, int lane) {
  constexpr int kPer = 16 / sizeof(T);           // columns a chunk
  constexpr int kChunks = kWords / 4;            // chunks a row: 4 or 8
  constexpr int kRows = mx4_round_rows(kWords);  // 32 or 16
  constexpr int kShift = kChunks == 4 ? 1 : 0;   // two rows of 64 bytes share a 128-byte line of the box
#pragma unroll
  for (int g = 0; g < 32 / kRows; ++g) {
    if (g * kRows >= valid) break;
    if (lane == 0) bulk_wait_read<0>();  // the store of the box's previous rows has read them
    __syncwarp();
    if (lane / kRows == g) {
      const int rr = lane % kRows;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        *reinterpret_cast<uint4*>(box + rr * 4 * kWords + ((j ^ ((rr >> kShift) & (kChunks - 1))) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
    if (p.align == 16 && (g + 1) * kRows <= valid && col + kChunks * kPer <= p.c_cols) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&p.tmC, box, col, row + g * kRows);
        bulk_commit();
      }
      continue;
    }
    __syncwarp();
    T* c = static_cast<T*>(p.c) + (long long)(row + g * kRows) * p.ldc + col;
    if (p.align == 16)
      mx4_store_units<4, kRows, kChunks, kShift>(box, c, p.ldc, p.c_cols - col, valid - g * kRows, lane);
    else if (kWords == 32 && p.align == 8)
      mx4_store_units<2, kRows, kChunks, kShift>(box, c, p.ldc, p.c_cols - col, valid - g * kRows, lane);
    else
      mx4_store_words<kRows, kChunks>(box, c, p.ldc, p.c_cols - col, valid - g * kRows, lane);
  }
}

template <typename T, bool GLU, int BN>
__global__ void __launch_bounds__(kMx4Threads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4GemmParams p) {
  using C = Mx4Cfg<BN>;
  constexpr int S = C::kStages;
  constexpr bool kOverlap = BN == 256;
  // the swizzled tiles need 1024-byte boundaries: dynamic shared memory begins on one where a kernel
  // has no static shared memory (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + S;
  uint64_t* sload = empty + S;  // the stage's scale atoms are in shared memory
  uint64_t* sfull = sload + S;  // ... and in TMEM
  uint64_t* tfull = sfull + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* tovl = tempty + 2;  // the shared columns of the tile before have been read
  uint64_t* drain = tovl + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&sload[i], 1);
      mbar_init(&sfull[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kMx4EpiWarps);
    }
    mbar_init(tovl, kMx4EpiWarps);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(&p.tmSA);
    tma_prefetch_desc(&p.tmSB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sf_base = tmem_base + C::kSfCols;
  pdl_wait();
  pdl_trigger();
  const Mx4Tiles tiles = mx4_tiles(p.rows, reinterpret_cast<int*>(smem + C::kTableOffset), p.status);
  int num_tiles = tiles.total * p.n_tiles;  // less than 2^31, as the host has seen to
  if (smem_u32(smem) & 1023u) {  // never so: no tile is touched, and the call reports it
    num_tiles = 0;
    if (threadIdx.x == 0) set_status(p.status, LMOE_STATUS_WATCHDOG);
  }
  const int split = BN == 128 ? p.split : 1;
  const int first = blockIdx.x / split;
  const int stride = gridDim.x / split;
  const int part = split > 1 ? (int)(blockIdx.x % split) : 0;
  const int kb0 = (int)((long long)p.nkb * part / split), kb1 = (int)((long long)p.nkb * (part + 1) / split);

  // row tile (of A, and so of its scales), its group, first row and valid rows, and tile of N of tile
  // `tile`, for a whole warp; N runs fastest, so the CTAs share few row tiles' rows and the weights of
  // few groups
  auto locate = [&](int tile, int& mt, int& g, int& row0, int& valid, int& nt) {
    mt = (unsigned)tile / (unsigned)p.n_tiles;
    nt = tile - mt * p.n_tiles;
    tiles.get(mt, g, row0, valid);
  };

  if (warp == 0) {
    // ---------------- loads (lane 0)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0, armed_parity = 0;
    bool ok = true;
    for (int tile = first; ok && tile < num_tiles; tile += stride) {
      int mt, g, row0, valid, nt;
      locate(tile, mt, g, row0, valid, nt);
      if (lane == 0) {
        const int brow0 = g * p.N + nt * BN;
        const int sb0 = g * p.b_tiles + nt * (BN / 128);
        // a tile of few rows loads 4 KB of A a k-block, not 16 (one token's 16 experts 7.6 us against 9.0,
        // 32 x 8192 x 7168 10.1 against 12.6)
        const bool few = valid <= 32;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort, p.status)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = smem + stage * C::kStageBytes;
          uint8_t* b_dst = a_dst + C::kABytes;
          uint8_t* s_dst = b_dst + C::kBBytes;
          // the scales first, on a barrier of their own: they are in TMEM before the tiles are here
          mbar_expect_tx(&sload[stage], 1024 + C::kSBBytes);
          tma_load_3d(s_dst, &p.tmSA, &sload[stage], 0, kb * 8, mt);
          tma_load_3d(s_dst + 1024, &p.tmSB, &sload[stage], 0, kb * 8, sb0);
          mbar_expect_tx(&full[stage], C::kABytes + C::kBBytes - (few ? 96 * 128 : 0));
          tma_load_2d(a_dst, few ? &p.tmA32 : &p.tmA, &full[stage], kb * 128, row0);
          tma_load_2d(b_dst, &p.tmB, &full[stage], kb * 128, brow0);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (!ok && lane == 0)
      for (int i = 0; i < S; ++i)
        if ((armed >> i) & 1u) {
          mbar_drain(&full[i], (armed_parity >> i) & 1u);
          mbar_drain(&sload[i], (armed_parity >> i) & 1u);
        }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int tile = first; ok && tile < num_tiles; tile += stride, ++it) {
        const int acc = it & 1;
        ok = mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, abort, p.status);
        if (kOverlap && ok && it) ok = mbar_wait(tovl, (it - 1) & 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * C::kAcc1;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort, p.status) || !mbar_wait(&sfull[stage], phase, abort, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * C::kStageBytes);
          const uint32_t b_addr = a_addr + C::kABytes;
          const uint32_t sfa = sf_base + stage * C::kSfBuf, sfb = sfa + 8;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_mxf4(d_tmem, smem_desc_sw128(a_addr + k * 32), smem_desc_sw128(b_addr + k * 32),
                        idesc_mxf4(BN, 128, 2 * (k & 1)), sfa + 4 * (k >> 1), sfb + (BN / 32) * (k >> 1),
                        (kb > kb0) | (k != 0));
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
  } else if (warp >= 10) {
    // ---------------- scales: warp w writes lane quarter w % 4 (all four hold the same words: lane i of
    // an atom's column j is the four scales of row i + 32 j).  Columns of a stage: A's atoms h = 0, 1
    // (columns [128 h, +128) of K) at 4 h, B's at 8 + (BN / 32) h, four for each 128 rows
    const uint32_t tq = sf_base + ((uint32_t)((warp & 3) * 32) << 16);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = first; ok && tile < num_tiles; tile += stride) {
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait(&sload[stage], phase, abort, p.status);
        __syncwarp();
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();  // the MMAs that last read these columns committed before the stage was loaded again
        const uint8_t* s_src = smem + stage * C::kStageBytes + C::kABytes + C::kBBytes + 16 * lane;
        const uint32_t t = tq + stage * C::kSfBuf;
        uint4 v[2 + BN / 64];
#pragma unroll
        for (int i = 0; i < 2 + BN / 64; ++i) v[i] = *reinterpret_cast<const uint4*>(s_src + 512 * i);
        tmem_st4(t, v[0]);
        tmem_st4(t + 4, v[1]);
#pragma unroll
        for (int j = 0; j < BN / 128; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) tmem_st4(t + 8 + (BN / 32) * h + 4 * j, v[2 + 2 * j + h]);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---------------- epilogue warps 2..9: TMEM lane quarter (warp % 4), column half (warp - 2) / 4
    const int wq = warp & 3;
    const int half_id = (warp - 2) >> 2;
    uint8_t* box = smem + C::kStgOffset + (warp - 2) * 2048;
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int it = 0;
    bool ok = true;
    for (int tile = first; ok && tile < num_tiles; tile += stride, ++it) {
      int mt, g, row0, valid, nt;
      locate(tile, mt, g, row0, valid, nt);
      const int acc = it & 1;
      ok = mbar_wait(&tfull[acc], (it >> 1) & 1, abort, p.status);
      __syncwarp();
      if (__any_sync(0xffffffffu, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(wq * 32) << 16) + acc * C::kAcc1;
      const int crow = row0 + wq * 32;
      const int vrows = valid - wq * 32;  // valid rows of this warp's 32
      if (split > 1) {
        // this CTA's part of the sum into the stages (every load has been consumed), rows 132 floats
        // apart: eight lanes' 16-byte stores then hit distinct banks
        float* parts = reinterpret_cast<float*>(smem) + (wq * 32 + lane) * kMx4PartPitch + half_id * 64;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t v[32];
          tmem_ld32(tbase + half_id * 64 + j * 32, v);
          tc_wait_ld();
          if (vrows > 0)
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(parts + j * 32 + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        tc_fence_before();
        continue;
      }
      // 128 columns at a time, the warp's half of them, those shared with the other accumulator (the
      // first accumulator's last 128, the second's first) before the others
      constexpr int kSteps = BN / 128;
#pragma unroll 1
      for (int j = 0; j < kSteps; ++j) {
        const int blk = kOverlap ? (j ^ acc ^ 1) : 0;
        // GLU: 64 gate and 64 linear columns, half h the features [32 h, +32) of them
        uint32_t v[2][32];
        tmem_ld32(tbase + blk * 128 + half_id * (GLU ? 32 : 64), v[0]);
        tmem_ld32(tbase + blk * 128 + (GLU ? 64 + half_id * 32 : 32 + half_id * 64), v[1]);
        tc_wait_ld();
        if (kOverlap && j == 0) arrive(tovl);
        if (j == kSteps - 1) arrive(&tempty[acc]);
        if constexpr (GLU) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = pack_bf16x2(silu_fast(__uint_as_float(v[0][2 * i])) * __uint_as_float(v[1][2 * i]),
                               silu_fast(__uint_as_float(v[0][2 * i + 1])) * __uint_as_float(v[1][2 * i + 1]));
          mx4_store_rows<16, T>(p, box, w, crow, nt * (BN / 2) + blk * 64 + half_id * 32, vrows, lane);
        } else {
          const int col = nt * BN + blk * 128 + half_id * 64;
          if constexpr (sizeof(T) == 4) {
            mx4_store_rows<32, T>(p, box, v[0], crow, col, vrows, lane);
            mx4_store_rows<32, T>(p, box, v[1], crow, col + 32, vrows, lane);
          } else {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              w[i] = pack_bf16x2(__uint_as_float(v[i >> 4][2 * (i & 15)]), __uint_as_float(v[i >> 4][2 * (i & 15) + 1]));
            mx4_store_rows<32, T>(p, box, w, crow, col, vrows, lane);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // every TMA store has left shared memory and landed
    if (p.zero_rest)
      mx4_zero_rest(tiles, p.rows.rows, static_cast<T*>(p.c), p.ldc, p.c_cols, blockIdx.x * kMx4EpiWarps + warp - 2,
                    gridDim.x * kMx4EpiWarps, lane);
  }

  if constexpr (BN == 128) {
    if (split > 1) {
      // the parts are added in their order; CTA r of the cluster takes the r-th share of the output
      // columns, a thread four of them of a row
      __syncthreads();
      cluster_sync_all();
      if (first < num_tiles && *abort == 0) {
        int mt, g, row0, valid, nt;
        locate(first, mt, g, row0, valid, nt);
        const uint32_t base = smem_u32(smem);
        constexpr int kCols = GLU ? 64 : 128;
        const int quads = kCols / 4 / split;  // split is 1, 2, 4 or 8
        for (int i = threadIdx.x; i < quads * valid; i += kMx4Threads) {
          const int r = i / quads, cc = ((i - r * quads) + part * quads) * 4;
          const int col = nt * kCols + cc;
          if (col >= p.c_cols) continue;
          const uint32_t at = base + (uint32_t)(r * kMx4PartPitch + cc) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
          for (int q = 0; q < split; ++q) {
            const uint32_t peer = mapa_shared(at, (uint32_t)q);
            add4(v, ld_shared_cluster4(peer));
            if constexpr (GLU) add4(u, ld_shared_cluster4(peer + 64 * 4));
          }
          float o[4] = {v.x, v.y, v.z, v.w};
          if constexpr (GLU) {
            o[0] = silu_fast(v.x) * u.x;
            o[1] = silu_fast(v.y) * u.y;
            o[2] = silu_fast(v.z) * u.z;
            o[3] = silu_fast(v.w) * u.w;
          }
          T* dst = static_cast<T*>(p.c) + (long long)(row0 + r) * p.ldc + col;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < p.c_cols) dst[j] = from_f<T>(o[j]);
        }
      }
      cluster_sync_all();  // no CTA leaves while its part is being read
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace lmoe
