// Host side of the entry points that need no layer handle and work on the caller's buffers: MXFP4
// quantisation, dequantisation and products, and the router's balance loss.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "balance.cuh"
#include "host.cuh"
#include "mx4_gemm.cuh"

using namespace lmoe;

namespace {

int device_sms(int* sms) {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LMOE_ECUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return LMOE_ECUDA;
  return major == 10 ? LMOE_OK : LMOE_EDEVICE;
}

// Row tiles the scale buffer has room for: ragged groups hold at most rows / 128 whole tiles and one
// partial tile each.
long long scale_tiles(int64_t rows, int32_t groups, bool ragged) {
  return ragged ? (rows + 127) / 128 + groups : (rows / groups + 127) / 128 * groups;
}
// Sizes of a matrix in groups.  The kernels count rows, and tiles x k-blocks x 8 slices, in 32 bits.
int check_rows(int64_t rows, int32_t cols, int32_t groups, bool ragged) {
  if (rows < 0 || cols <= 0 || groups <= 0) return LMOE_EINVAL;
  if (!ragged && rows % groups) return LMOE_EINVAL;
  if (cols % 32 || groups > kMx4MaxGroups || rows > (1ll << 30)) return LMOE_EUNSUPPORTED;
  if (scale_tiles(rows, groups, ragged) * mx4_kblocks(cols) * 8 >= (1ll << 31)) return LMOE_EUNSUPPORTED;
  return LMOE_OK;
}
// Row tiles a call can have: a group without rows has none.
long long work_tiles(int64_t rows, int32_t groups, bool ragged) {
  return ragged ? rows / 128 + std::min<int64_t>(groups, rows) : scale_tiles(rows, groups, false);
}

// Words the kernels read or add to: not null (unless it may be), on a 4-byte boundary.
bool words(const void* p, bool optional = false) { return (p || optional) && ((uintptr_t)p & 3) == 0; }

// Widest access that every row of a matrix allows (rows `ld` elements apart).
int row_access(const void* p, int64_t ld, int32_t dtype) {
  const uint64_t a = (uint64_t)(uintptr_t)p | (uint64_t)(ld * (dtype == LMOE_F32 ? 4 : 2));
  return a % 32 == 0 ? MX4_32 : (a % 16 == 0 ? MX4_16 : MX4_ELEMENTS);
}

// Grid of the quantisation kernels (eight warps a block, a block a tile and k-block at a time): at most
// 32 blocks an SM, so that what each does is even (eight cost dequantising a tenth more).
int mx4_grid(long long tiles, int nkb, int sms) { return (int)std::min(tiles * nkb, 32ll * sms); }

// Tensor map of a matrix's scale atoms: `tiles` row tiles of nkb k-blocks of 1 KB (two atoms), as rows of
// 128 bytes; a box is one k-block of `box_tiles` row tiles.
bool make_map_atoms(CUtensorMap* m, const uint8_t* scales, long long tiles, int nkb, int box_tiles) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || tiles <= 0) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)nkb * 8, (cuuint64_t)tiles};
  cuuint64_t strides[2] = {128, (cuuint64_t)nkb * 1024};
  cuuint32_t box[3] = {128, 8, (cuuint32_t)box_tiles};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(scales), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of a product's result: boxes of one staging round, rows of `words` words (64 bytes: 64-byte
// swizzle, 128: 128-byte).
bool make_map_c(CUtensorMap* m, void* c, long long rows, int cols, long long ld, bool f32, int words) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int es_bytes = f32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * es_bytes)};
  cuuint32_t box[2] = {(cuuint32_t)(4 * words / es_bytes), (cuuint32_t)mx4_round_rows(words)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, words == 16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool GLU, int BN>
int launch_mx4_gemm(const Mx4GemmParams& p, int grid, cudaStream_t st) {
  auto kern = mx4_gemm_kernel<T, GLU, BN>;
  static unsigned done = 0;
  constexpr int smem = Mx4Cfg<BN>::kSmemBytes;
  CK(ensure_smem_attr(kern, smem, done));
  CK(launch_k(kern, dim3(grid), dim3(kMx4Threads), smem, st, p.split, p));
  return LMOE_OK;
}

// How a product is cut (see mx4_gemm.cuh): tile width, CTAs a tile, grid.
struct Mx4Plan {
  int bn, split, grid;
};
Mx4Plan plan_mx4(int M, int N, int nkb, int groups, bool ragged, int sms) {
  const long long mt = work_tiles(M, groups, ragged);
  const long long t128 = mt * ((N + 127) / 128), t256 = mt * ((N + 255) / 256);
  // 256-wide tiles where they take at most two thirds of the 128-wide ones' waves: 2048 x 2048 x 2048,
  // one wave for two, 8.1 us against 10.6; 16384 x 8192 x 7168 356 against 560; one token's 16 experts,
  // one wave either way, 8.8 against 7.8
  if ((t256 + sms - 1) / sms * 3 <= (t128 + sms - 1) / sms * 2)
    return {256, 1, (int)std::min<long long>(t256, sms)};
  // too few tiles for the GPU and a K of 12 k-blocks or more: clusters share the tiles (1 x 1024 x 7168
  // 12.0 us alone, 7.0 in fours, 6.3 in eights; 1 x 7168 x 2048, eight k-blocks, 6.2 alone, 6.5 in twos).
  // Eight CTAs only while half the GPU holds them all, since not every SM has seven neighbours free
  // (16 tiles of 2048 x 4096: 19.6 us in eights, 8.5 in fours)
  int split = 1;
  if (nkb >= 12)
    while (split < 8 && nkb >= 8 * split && 2 * split * t128 <= (split < 4 ? sms : sms / 2)) split *= 2;
  return {128, split, (int)std::min<long long>(t128 * split, sms)};
}

// The balance loss in one launch (a cluster) or two (see balance.cuh).
template <int NJ, int VEC, int R, int LANES>
int launch_balance(BalanceParams& p, int sms, cudaStream_t st, long long* launches) {
  constexpr int kRound = kBalThreads / LANES * R;  // rows of one round of a block
  // One launch where a cluster streams the scores about as fast as the GPU gets through two launches
  // more (2048 x 256: 13.5 and 12.5 us on the GPU, 16 and 19.5 us with the host's launches; 512 x 64:
  // 6.9 and 10.5; 4096 x 256: 19 and 13): 2^15 scores a CTA of the largest cluster
  const bool fits = (long long)p.S * p.E <= kBalHistInts;  // the cluster form's shared counters
  auto kern = balance_cluster_kernel<NJ, VEC, R, LANES>;
  static std::atomic<unsigned> known{0}, large{0};
  const int most = fits ? largest_cluster(kern, kBalThreads, known, large) : 0;
  if ((long long)p.T * p.E <= (long long)most << 15) {
    const int ctas = bal_ctas(p.T, p.S, kRound, most);
    p.chunk = (p.T + ctas - 1) / ctas;
    CK(launch_k(kern, dim3(ctas), dim3(kBalThreads), 0, st, ctas, p));
    if (launches) *launches += 1;
    return LMOE_OK;
  }
  CK(cudaMemsetAsync(p.counts, 0, (size_t)p.S * p.E * sizeof(int32_t), st));
  // counting: runs of some 64 tokens, fewer where the sequences are shorter (a block takes its sequences in
  // turn), at most a block an SM
  const int per_seq = (p.T + p.S - 1) / p.S;
  p.chunk = std::max(std::min(64, per_seq), (p.T + sms - 1) / sms);
  CK(launch_k(balance_count_kernel, dim3((p.T + p.chunk - 1) / p.chunk), dim3(kBalThreads), 0, st, 1, p));
  // the pass: one round of rows a block, or a sequence, at most the two blocks an SM that its registers allow
  const int blocks = std::min(2 * sms, kBalMaxBlocks);
  p.chunk = std::max(std::min(kRound, per_seq), (p.T + blocks - 1) / blocks);
  CK(launch_k(balance_kernel<NJ, VEC, R, LANES>, dim3((p.T + p.chunk - 1) / p.chunk), dim3(kBalThreads), 0, st, 1, p));
  if (launches) *launches += 2;
  return LMOE_OK;
}

}  // namespace

int lmoe::balance_loss(const float* scores, const int32_t* idx, int32_t T, int32_t E, int32_t k,
                       const int32_t* cu_seqlens, int32_t S, const int32_t* total, float coef, int32_t* counts,
                       float* loss, float* dscores, void* scratch, uint32_t* status, void* stream,
                       long long* launches) {
  if (T < 0 || E <= 0 || k <= 0 || k > E || S <= 0 || (!cu_seqlens && S != 1) || !(coef == coef)) return LMOE_EINVAL;
  if (E > kBalMaxE || k > 32 || S > kBalMaxSeqs || (long long)T * k > (1ll << 30)) return LMOE_EUNSUPPORTED;
  if (!words(counts) || !words(loss) || !words(status) || !scratch || ((uintptr_t)scratch & 15)) return LMOE_EINVAL;
  if (!words(scores, T == 0) || !words(idx, T == 0) || !words(dscores, true) || !words(cu_seqlens, true))
    return LMOE_EINVAL;
  int sms = 0;
  const int rc = device_sms(&sms);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) {
    CK(cudaMemsetAsync(counts, 0, (size_t)S * E * sizeof(int32_t), st));
    CK(cudaMemsetAsync(loss, 0, sizeof(float), st));
    return LMOE_OK;
  }
  BalanceParams p;
  memset(&p, 0, sizeof(p));
  p.scores = scores;
  p.idx = idx;
  p.cu = cu_seqlens;
  p.T = T;
  p.E = E;
  p.k = k;
  p.S = S;
  p.total = total;
  p.coef = coef;
  p.counts = counts;
  p.loss = loss;
  p.dscores = dscores;
  p.done = static_cast<unsigned*>(scratch);
  p.partial = reinterpret_cast<double*>(static_cast<char*>(scratch) + 256);
  p.status = status;
  const bool vec = E % 4 == 0 && (((uintptr_t)scores | (uintptr_t)dscores) & 15) == 0;
  // sets of rows in flight: what fits the 64 registers that two blocks an SM leave a thread; rows of few
  // experts share a warp (262144 x 8 19 us against 39 with a row a warp, 65536 x 64 15 against 19)
  if (vec) {
    if (E <= 32) return launch_balance<1, 4, 4, 8>(p, sms, st, launches);
    if (E <= 64) return launch_balance<1, 4, 4, 16>(p, sms, st, launches);
    if (E <= 128) return launch_balance<1, 4, 4, 32>(p, sms, st, launches);
    if (E <= 256) return launch_balance<2, 4, 4, 32>(p, sms, st, launches);
    if (E <= 512) return launch_balance<4, 4, 2, 32>(p, sms, st, launches);
    return launch_balance<8, 4, 2, 32>(p, sms, st, launches);
  }
  if (E <= 64) return launch_balance<2, 1, 4, 32>(p, sms, st, launches);
  if (E <= 256) return launch_balance<8, 1, 4, 32>(p, sms, st, launches);
  return launch_balance<32, 1, 1, 32>(p, sms, st, launches);
}

extern "C" {

int lmoe_mx4_bytes(int64_t rows, int32_t cols, int32_t groups, int32_t ragged, size_t* elem_bytes,
                   size_t* scale_bytes) {
  const int rc = check_rows(rows, cols, groups, ragged != 0);
  if (rc) return rc;
  if (!elem_bytes || !scale_bytes) return LMOE_EINVAL;
  *elem_bytes = (size_t)rows * (cols / 2);
  *scale_bytes = (size_t)scale_tiles(rows, groups, ragged != 0) * mx4_kblocks(cols) * 1024;
  return LMOE_OK;
}

int lmoe_mx4_quant(const void* x, int32_t dtype, int64_t ld, const int32_t* index, int64_t x_rows, int64_t rows,
                   int32_t cols, int32_t groups, const int32_t* offsets, uint8_t* elems, uint8_t* scales,
                   uint32_t* status, void* stream) {
  const int rc = check_rows(rows, cols, groups, offsets != nullptr);
  if (rc) return rc;
  if (dtype != LMOE_F32 && dtype != LMOE_BF16) return LMOE_EINVAL;
  if (index && (x_rows < 0 || x_rows > INT32_MAX)) return LMOE_EINVAL;
  if (rows == 0) return LMOE_OK;
  if (!x && !(index && x_rows == 0)) return LMOE_EINVAL;  // every index is outside an x without rows
  if (!elems || !scales || ld < cols || ((uintptr_t)elems & 15) || ((uintptr_t)scales & 15)) return LMOE_EINVAL;
  if (!words(status) || !words(offsets, true) || !words(index, true)) return LMOE_EINVAL;
  if ((uintptr_t)x % (dtype == LMOE_F32 ? 4 : 2)) return LMOE_EINVAL;
  int sms = 0;
  const int drc = device_sms(&sms);
  if (drc) return drc;
  Mx4QuantParams p;
  memset(&p, 0, sizeof(p));
  p.src = x;
  p.index = index;
  p.src_rows = (int)x_rows;
  p.ld = ld;
  p.cols = cols;
  p.rows = Mx4Rows{offsets, groups, (int)rows};
  p.elems = elems;
  p.scales = scales;
  p.status = status;
  p.access = row_access(x, ld, dtype);
  const int grid = mx4_grid(work_tiles(rows, groups, offsets != nullptr), mx4_kblocks(cols), sms);
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 g(grid), b(256);
  if (index) {
    if (dtype == LMOE_F32) CK(launch_k(mx4_quant_kernel<float, MX4_INDEXED>, g, b, 0, st, 1, p));
    else CK(launch_k(mx4_quant_kernel<bf16, MX4_INDEXED>, g, b, 0, st, 1, p));
  } else {
    if (dtype == LMOE_F32) CK(launch_k(mx4_quant_kernel<float, MX4_PLAIN>, g, b, 0, st, 1, p));
    else CK(launch_k(mx4_quant_kernel<bf16, MX4_PLAIN>, g, b, 0, st, 1, p));
  }
  return LMOE_OK;
}

int lmoe_mx4_quant_w13(const void* w1, const void* w3, int32_t dtype, int32_t groups, int32_t h, int32_t cols,
                       uint8_t* elems, uint8_t* scales, uint32_t* status, void* stream) {
  if (h <= 0 || groups <= 0) return LMOE_EINVAL;
  if (h % 64) return LMOE_EUNSUPPORTED;
  const int64_t rows = 2ll * groups * h;
  const int rc = check_rows(rows, cols, groups, false);
  if (rc) return rc;
  if (dtype != LMOE_F32 && dtype != LMOE_BF16) return LMOE_EINVAL;
  if (!w1 || !w3 || !elems || !scales || !words(status) || ((uintptr_t)elems & 15) || ((uintptr_t)scales & 15))
    return LMOE_EINVAL;
  if (((uintptr_t)w1 | (uintptr_t)w3) % (dtype == LMOE_F32 ? 4 : 2)) return LMOE_EINVAL;
  int sms = 0;
  const int drc = device_sms(&sms);
  if (drc) return drc;
  Mx4QuantParams p;
  memset(&p, 0, sizeof(p));
  p.src = w1;
  p.src3 = w3;
  p.ld = cols;
  p.cols = cols;
  p.rows = Mx4Rows{nullptr, groups, (int)rows};
  p.elems = elems;
  p.scales = scales;
  p.status = status;
  p.access = std::min(row_access(w1, cols, dtype), row_access(w3, cols, dtype));
  const int grid = mx4_grid(work_tiles(rows, groups, false), mx4_kblocks(cols), sms);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == LMOE_F32)
    CK(launch_k(mx4_quant_kernel<float, MX4_PAIRED>, dim3(grid), dim3(256), 0, st, 1, p));
  else
    CK(launch_k(mx4_quant_kernel<bf16, MX4_PAIRED>, dim3(grid), dim3(256), 0, st, 1, p));
  return LMOE_OK;
}

int lmoe_mx4_dequant(const uint8_t* elems, const uint8_t* scales, int64_t rows, int32_t cols, int32_t groups,
                     const int32_t* offsets, void* out, int32_t dtype, int64_t ld, uint32_t flags, uint32_t* status,
                     void* stream) {
  const int rc = check_rows(rows, cols, groups, offsets != nullptr);
  if (rc) return rc;
  if ((dtype != LMOE_F32 && dtype != LMOE_BF16) || (flags & ~LMOE_MX4_ZERO_REST)) return LMOE_EINVAL;
  if (rows == 0) return LMOE_OK;
  if (!out || !elems || !scales || ld < cols || ((uintptr_t)elems & 15) || ((uintptr_t)scales & 15)) return LMOE_EINVAL;
  if (!words(status) || !words(offsets, true)) return LMOE_EINVAL;
  if ((uintptr_t)out % (dtype == LMOE_F32 ? 4 : 2)) return LMOE_EINVAL;
  int sms = 0;
  const int drc = device_sms(&sms);
  if (drc) return drc;
  Mx4DequantParams p;
  memset(&p, 0, sizeof(p));
  p.elems = elems;
  p.scales = scales;
  p.out = out;
  p.ld = ld;
  p.cols = cols;
  p.rows = Mx4Rows{offsets, groups, (int)rows};
  p.status = status;
  p.zero_rest = (flags & LMOE_MX4_ZERO_REST) ? 1 : 0;
  p.access = row_access(out, ld, dtype);
  const int grid = mx4_grid(work_tiles(rows, groups, offsets != nullptr), mx4_kblocks(cols), sms);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == LMOE_F32)
    CK(launch_k(mx4_dequant_kernel<float>, dim3(grid), dim3(256), 0, st, 1, p));
  else
    CK(launch_k(mx4_dequant_kernel<bf16>, dim3(grid), dim3(256), 0, st, 1, p));
  return LMOE_OK;
}

int lmoe_mx4_gemm(const uint8_t* a_elems, const uint8_t* a_scales, const uint8_t* b_elems, const uint8_t* b_scales,
                  int32_t M, int32_t N, int32_t K, int32_t groups, const int32_t* offsets, void* c, int32_t c_dtype,
                  int64_t ldc, uint32_t flags, uint32_t* status, void* stream) {
  if (M < 0 || N <= 0 || K <= 0 || groups <= 0) return LMOE_EINVAL;
  if ((groups > 1 && !offsets) || (flags & ~(LMOE_MX4_SWIGLU | LMOE_MX4_ZERO_REST))) return LMOE_EINVAL;
  const bool swiglu = (flags & LMOE_MX4_SWIGLU) != 0;
  if (c_dtype != LMOE_F32 && c_dtype != LMOE_BF16) return LMOE_EINVAL;
  int rc = check_rows(M, K, groups, offsets != nullptr);
  if (!rc) rc = check_rows((int64_t)groups * N, K, groups, false);
  if (rc) return rc;
  if (scale_tiles(M, groups, offsets != nullptr) * ((N + 127) / 128) >= (1ll << 31)) return LMOE_EUNSUPPORTED;
  if (swiglu && (N % 128 || c_dtype != LMOE_BF16)) return LMOE_EUNSUPPORTED;
  if (M == 0) return LMOE_OK;
  const int32_t cols = swiglu ? N / 2 : N;
  if (!a_elems || !a_scales || !b_elems || !b_scales || !c || ldc < cols) return LMOE_EINVAL;
  if (!words(status) || !words(offsets, true)) return LMOE_EINVAL;
  if (((uintptr_t)a_elems | (uintptr_t)a_scales | (uintptr_t)b_elems | (uintptr_t)b_scales) & 15) return LMOE_EINVAL;
  if ((uintptr_t)c % (c_dtype == LMOE_F32 ? 4 : 2)) return LMOE_EINVAL;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc) return rc;
  const int nkb = mx4_kblocks(K);
  const Mx4Plan plan = plan_mx4(M, N, nkb, groups, offsets != nullptr, sms);
  Mx4GemmParams p;
  memset(&p, 0, sizeof(p));
  p.b_tiles = (N + 127) / 128;
  if (!make_map_u8(&p.tmA, a_elems, M, K / 2, K / 2, 128) || !make_map_u8(&p.tmA32, a_elems, M, K / 2, K / 2, 32) ||
      !make_map_u8(&p.tmB, b_elems, (long long)groups * N, K / 2, K / 2, plan.bn) ||
      !make_map_atoms(&p.tmSA, a_scales, scale_tiles(M, groups, offsets != nullptr), nkb, 1) ||
      !make_map_atoms(&p.tmSB, b_scales, (long long)groups * p.b_tiles, nkb, plan.bn / 128))
    return LMOE_ECUDA;
  p.rows = Mx4Rows{offsets, groups, M};
  p.N = N;
  p.n_tiles = (N + plan.bn - 1) / plan.bn;
  p.nkb = nkb;
  p.split = plan.split;
  p.c = c;
  p.ldc = ldc;
  p.c_cols = cols;
  p.zero_rest = (flags & LMOE_MX4_ZERO_REST) ? 1 : 0;
  p.align = 16;
  while (((uint64_t)(uintptr_t)c | (uint64_t)ldc * (c_dtype == LMOE_F32 ? 4 : 2)) & (p.align - 1)) p.align /= 2;
  p.status = status;
  if (p.align == 16 && !make_map_c(&p.tmC, c, M, cols, ldc, c_dtype == LMOE_F32, swiglu ? 16 : 32)) return LMOE_ECUDA;
  cudaStream_t st = (cudaStream_t)stream;
  auto launch = [&](auto type, auto glu) -> int {
    using T = decltype(type);
    constexpr bool G = decltype(glu)::value;
    if (plan.bn == 256) return launch_mx4_gemm<T, G, 256>(p, plan.grid, st);
    return launch_mx4_gemm<T, G, 128>(p, plan.grid, st);
  };
  if (swiglu) return launch(bf16(), std::true_type());
  if (c_dtype == LMOE_BF16) return launch(bf16(), std::false_type());
  return launch(0.f, std::false_type());
}

int lmoe_balance_scratch_bytes(size_t* bytes) {
  if (!bytes) return LMOE_EINVAL;
  *bytes = kBalMaxBlocks * sizeof(double) + 256;
  return LMOE_OK;
}

int lmoe_balance_loss(const float* scores, const int32_t* idx, int32_t T, int32_t E, int32_t k,
                      const int32_t* cu_seqlens, int32_t S, float coef, int32_t* counts, float* loss, float* dscores,
                      void* scratch, uint32_t* status, void* stream) {
  return balance_loss(scores, idx, T, E, k, cu_seqlens, S, nullptr, coef, counts, loss, dscores, scratch, status,
                      stream, nullptr);
}

}  // extern "C"
