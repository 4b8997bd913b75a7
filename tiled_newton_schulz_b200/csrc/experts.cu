// experts.cu -- products over row groups: expert forward and input-gradient
// products, weight gradients and the 8-bit product (checks, tensor maps, launches).
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <atomic>
#include <vector>

#include "experts_kernel.cuh"
#include "layout.hpp"

namespace himuon {

// SMs of the current device (looked up once per device).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p)
               : nullptr;
  }();
  return fn;
}

// Map over `n` row-major matrices `stride` bytes apart (2-D when n = 0): boxes
// of box_rows x box_cols (0: as many as make 128 bytes) with the swizzle of the
// box's width (64 or 128 bytes), zeros outside.
bool make_map(CUtensorMap *map, const himuon_mat &m, int32_t n, int64_t stride, uint32_t box_rows,
              uint32_t box_cols = 0) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t es = static_cast<int64_t>(size_of(m.dtype));
  if (!box_cols) box_cols = static_cast<uint32_t>(128 / es);
  const CUtensorMapDataType dt = m.dtype == HIMUON_I8     ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : m.dtype == HIMUON_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : m.dtype == HIMUON_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // the pitch of a single row is never used and may be any number
  const int64_t pitch = m.rows > 1 ? m.ld * es : (m.cols * es + 15) / 16 * 16;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows),
                        static_cast<cuuint64_t>(n > 0 ? n : 1)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(n > 1 ? stride : pitch * m.rows)};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t es1[3] = {1, 1, 1};
  return enc(map, dt, n > 0 ? 3 : 2, m.data, dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row operand as overlapping windows: coordinates (column, r, row) are row `row`
// + r, r < 64, so that a box that begins at r = left - 64 holds 64 - left rows of
// zeros and then rows row .. row + left - 1.
bool make_window_map(CUtensorMap *map, const himuon_mat &m) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t es = static_cast<int64_t>(size_of(m.dtype));
  const CUtensorMapDataType dt =
      m.dtype == HIMUON_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t pitch = static_cast<cuuint64_t>(m.rows > 1 ? m.ld * es : (m.cols * es + 15) / 16 * 16);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), 64, static_cast<cuuint64_t>(m.rows)};
  cuuint64_t strides[2] = {pitch, pitch};
  cuuint32_t box[3] = {64, 64, 1};
  cuuint32_t es1[3] = {1, 1, 1};
  return enc(map, dt, 3, m.data, dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Do the matrices lie one behind the other at equal distances, a multiple of
// their pitch in a tensor map's range?  `stride`: that distance.  (Anything else,
// such as column blocks of one fused matrix, runs as a list.)
bool stacked(const himuon_mat *m, int32_t n, int64_t *stride) {
  *stride = 0;
  if (n == 1) return true;
  const int64_t d = static_cast<const char *>(m[1].data) - static_cast<const char *>(m[0].data);
  const int64_t pitch = m->ld * static_cast<int64_t>(size_of(m->dtype));
  if (d < pitch * m->rows || d % pitch != 0 || pitch % 16 != 0 || d >= (int64_t)1 << 39) return false;
  for (int32_t e = 1; e < n; ++e)
    if (static_cast<const char *>(m[e].data) - static_cast<const char *>(m[e - 1].data) != d) return false;
  *stride = d;
  return true;
}

// Loads both list forms of a variant of the kernel, allows them their shared memory
// and sees to it that they are launched with the registers that they move.
template <int KIND, int A_MN, int GRAD, int PREC, int SPLIT>
bool load_variant() {
  auto load = [](auto kern) {
    cudaFuncAttributes f;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
           cudaFuncGetAttributes(&f, kern) == cudaSuccess &&
           (!kMovesRegisters<GRAD, PREC, SPLIT> || f.numRegs >= kRegsLaunch);
  };
  return load(expert_kernel<KIND, A_MN, GRAD, 1, 1, PREC, SPLIT>) &&
         load(expert_kernel<KIND, A_MN, GRAD, GRAD ? 1 : kMaxList, GRAD ? kMaxList : 1, PREC, SPLIT>);
}
// How many clusters of `split` pairs run at once: fewer than the pairs would
// make, since a cluster lives inside one of the device's processor clusters
// (148 SMs hold 74 pairs, but not 37 clusters of four SMs or 18 of eight).
// A property of the device; 0 if it cannot be had.
std::atomic<int32_t> cluster_room[64][2];
int32_t clusters_at_once(int32_t split) {
  if (split == 1) return sm_count() / 2;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int32_t> *known = dev < 64 ? &cluster_room[dev][split / 4] : nullptr;
  if (known && known->load(std::memory_order_relaxed)) return known->load(std::memory_order_relaxed);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2 * split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int room = 0;
  if (cudaOccupancyMaxActiveClusters(&room, expert_kernel<0, 0, 0, 1, 1, 1, 1>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (known) known->store(room, std::memory_order_relaxed);
  return room;
}
bool load_kernels() {
  static std::atomic<uint64_t> loaded{0};   // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (loaded.load(std::memory_order_relaxed) & bit) return true;
  const bool ok =
      load_variant<0, 0, 0, 0, 0>() && load_variant<0, 0, 0, 1, 0>() && load_variant<0, 0, 0, 2, 0>() &&
      load_variant<0, 0, 0, 1, 1>() && load_variant<0, 1, 0, 2, 0>() &&
      load_variant<0, 1, 0, 0, 0>() && load_variant<0, 1, 0, 1, 0>() && load_variant<0, 1, 0, 1, 1>() &&
      load_variant<1, 0, 0, 0, 0>() && load_variant<1, 0, 0, 1, 1>() && load_variant<0, 1, 1, 0, 0>() &&
      load_variant<0, 1, 1, 1, 0>() && load_variant<0, 1, 1, 1, 1>() && device_status_word() != nullptr &&
      load_quantize();
  clusters_at_once(2);   // (looked up here, not in a later call's capture; with no room, tiles are not shared)
  clusters_at_once(4);
  if (ok) loaded.fetch_or(bit, std::memory_order_relaxed);
  return ok;
}
template <int KIND, int A_MN, int GRAD, int PREC, int SPLIT, int NMAP, int NOUT>
int launch_mma(const MmaArgs<NMAP, NOUT> &a, int64_t most_tiles, cudaStream_t stream) {
  auto kern = expert_kernel<KIND, A_MN, GRAD, NMAP, NOUT, PREC, SPLIT>;
  const unsigned ctas = 2 * static_cast<unsigned>(a.split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * static_cast<unsigned>(SPLIT ? most_tiles : std::min<int64_t>(most_tiles, sm_count() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HIMUON_OK : HIMUON_ERR_CUDA;
}

// What a call of `tiles` tiles costs, in blocks of the sum, if `split` pairs (1, 2
// or 4) share a tile of `blocks` and `room` tiles run at once: the rounds, times a
// pair's share and `join` for starting the clusters and adding up.  Shared tiles
// run in one round only: a second would start its clusters anew (3 rows, 20000 ->
// 10240, bf16: 72 us with one pair per tile, 92 with four in three rounds).
int64_t split_cost(int64_t tiles, int64_t blocks, int32_t split, int64_t room, int64_t join) {
  if (room < 1 || (split > 1 && tiles > room)) return INT64_MAX;
  return (tiles + room - 1) / room * ((blocks + split - 1) / split + join);
}

template <int NMAP, int NOUT>
void common_args(MmaArgs<NMAP, NOUT> &a, const int32_t *offsets, int32_t e0, int32_t n, int64_t rows) {
  a.offsets = offsets ? offsets + e0 : nullptr;
  a.rows = rows;
  a.n = n;
  a.status = device_status_word();
  a.x_scale = a.w_scale = nullptr;
  a.ld_scale = 0;
  a.has_c = 0;
  a.ldo = a.out_stride = 0;
  a.buffers = 1;
  a.box_cols = 0;
  a.split = 1;
  a.least = 0;
  a.most = INT32_MAX;
  // HIMUON_TEST_STALL=1 exercises the device timeout path (tests only)
  const char *stall = getenv("HIMUON_TEST_STALL");
  a.stall = stall && stall[0] == '1';
  a.cdtype = HIMUON_BF16;
  a.alpha = 1.f;
  a.beta = 0.f;
}

// D format and operand formats of the instruction descriptor (its N field is
// set per tile): f32 from bf16/fp16, or s32 from s8.
uint32_t idesc_of(int32_t dtype, uint32_t a_mn, uint32_t b_mn) {
  if (dtype == HIMUON_I8) return (2u << 4) | (1u << 7) | (1u << 10) | ((kTileM >> 4) << 24);
  return idesc_f16(kTileM, 0, dtype == HIMUON_FP16 ? 0u : 1u, a_mn, b_mn, 0);
}

template <int NMAP>
int product_launch(const himuon_mat *X, const float *x_scale, const himuon_mat *W, int64_t stride,
                   const himuon_mat *w_scale, int32_t e0, int32_t n, const int32_t *offsets, int32_t w_trans,
                   const himuon_mat *Y, cudaStream_t stream) {
  MmaArgs<NMAP, 1> a;
  common_args(a, offsets, e0, n, X->rows);
  const uint32_t w_rows = w_trans ? 128 : 64;
  for (int32_t i = 0; i < (NMAP > 1 ? n : 1); ++i)
    if (!make_map(&a.w[i], W[e0 + i], NMAP > 1 ? 1 : n, stride, w_rows)) return HIMUON_ERR_CUDA;
  // (boxes of more rows than half of the widest tile are never loaded)
  const int64_t half = (std::min<int64_t>(X->rows, kTileN) + 31) / 32 * 16;
  for (int i = 0; i < 4; ++i)
    if ((128 >> i) <= half && !make_map(&a.x[i], *X, 0, 0, 128 >> i)) return HIMUON_ERR_CUDA;
  a.K = static_cast<int32_t>(X->cols);
  a.M = static_cast<int32_t>(Y->cols);
  a.N = 0;
  a.idesc = idesc_of(X->dtype, w_trans ? 0 : 1, 0);
  if (x_scale) {
    a.x_scale = x_scale;
    a.w_scale = static_cast<const float *>(w_scale->data) + e0 * w_scale->ld;
    a.ld_scale = w_scale->ld;
  }
  if (Y->dtype == HIMUON_FP32 && !make_map(&a.g[0], *Y, 0, 0, 16, 32)) return HIMUON_ERR_CUDA;
  a.out[0] = static_cast<char *>(Y->data);
  a.ldo = Y->ld;
  a.odtype = Y->dtype;
  // Row tiles of up to 256 rows move the fewest bytes.  Where even tiles of up to
  // 128 (below that a tile's loads of W bound it) cannot fill the pairs once,
  // whatever the groups' sizes, they are taken, and what pairs are left then
  // share the tiles' sums.  (One group of 512 rows, 4096 -> 4096: 28.7 us
  // with 256 rows, 20.5 with 128; where the cap lengthens the last round instead,
  // it costs: 1024 rows 28.7 us with 256, 32.9 with 128.)
  const int64_t mt_m = (Y->cols + kTileM - 1) / kTileM, pairs = sm_count() / 2;
  auto most_tiles = [&](int64_t cap) {
    return mt_m * (n == 1 ? (X->rows + cap - 1) / cap : X->rows / cap + std::min<int64_t>(n, X->rows));
  };
  a.cap = most_tiles(128) <= pairs ? 7 : 8;
  const int64_t most = most_tiles(1 << a.cap);
  a.mt_m = static_cast<int32_t>(mt_m);
  a.mt_n = 0;
  // Pairs share tiles where that is the shortest.  (A row, bf16, one pair, two and
  // four per tile: 4096 -> 4096, 16 tiles, 16.6, 13.1 and 20.2 us, since 16 clusters
  // of eight SMs do not run at once; 14336 -> 1024 44.5, 27.7 and 17.8; 1024 -> 4096
  // 8.4, 8.8 and 16.6.)
  if (a.cap == 7 || X->rows <= 128) {
    const int64_t blocks = (X->cols * static_cast<int64_t>(size_of(X->dtype)) + 127) / 128;
    int64_t best = split_cost(most, blocks, 1, pairs, 0);
    for (int32_t s = 2; s <= 4; s *= 2) {
      const int64_t cost = split_cost(most, blocks, s, clusters_at_once(s), s == 2 ? 12 : 16);
      if (cost >= best) continue;
      best = cost;
      a.split = s;
    }
  }
  const bool fp32 = Y->dtype == HIMUON_FP32, pieces = X->cols > 1 << longest_log(Y->dtype);
  a.piece_log = piece_log(X->cols, a.split > 1 ? HIMUON_FP32 : Y->dtype);
  if (X->dtype == HIMUON_I8)
    return a.split > 1 ? launch_mma<1, 0, 0, 1, 1>(a, most, stream) : launch_mma<1, 0, 0, 0, 0>(a, most, stream);
  if (w_trans)
    return a.split > 1 ? launch_mma<0, 0, 0, 1, 1>(a, most, stream)
           : fp32      ? launch_mma<0, 0, 0, 1, 0>(a, most, stream)
           : pieces    ? launch_mma<0, 0, 0, 2, 0>(a, most, stream)
                       : launch_mma<0, 0, 0, 0, 0>(a, most, stream);
  return a.split > 1 ? launch_mma<0, 1, 0, 1, 1>(a, most, stream)
         : fp32      ? launch_mma<0, 1, 0, 1, 0>(a, most, stream)
         : pieces    ? launch_mma<0, 1, 0, 2, 0>(a, most, stream)
                     : launch_mma<0, 1, 0, 0, 0>(a, most, stream);
}

int run_product(const himuon_mat *X, const float *x_scale, const himuon_mat *W, const himuon_mat *w_scale, int32_t n,
                const int32_t *offsets, int32_t w_trans, const himuon_mat *Y, cudaStream_t stream) {
  if (X->rows == 0) return HIMUON_OK;
  int64_t stride;
  const bool st = stacked(W, n, &stride);
  const int32_t cap = st ? kMaxStack : kMaxList;
  for (int32_t e0 = 0; e0 < n; e0 += cap) {
    const int32_t cnt = std::min(n - e0, cap);
    const int rc = st ? product_launch<1>(X, x_scale, W, stride, w_scale, e0, cnt, offsets, w_trans, Y, stream)
                      : product_launch<kMaxList>(X, x_scale, W, 0, w_scale, e0, cnt, offsets, w_trans, Y, stream);
    if (rc) return rc;
  }
  return HIMUON_OK;
}

// A gradient's tiles: their columns, how many lie across G, and the pairs that share
// one.  As few as 256 columns allow, or up to four times as many of equal width, in
// whole boxes of the epilogue, where that fills the last round of the pairs better.
// A block of the sum costs a pair the tile's columns, 128 at least, and as much as
// 192 more (0.20 us at up to 128 columns, 0.22 at 192, 0.29 at 256).  (bf16, 14808
// rows 64 x 1408: one tile per pair 48.7 us at 128 columns, four pairs per tile 22.0;
// 8192 rows 1024 x 1024 31.4, and 25.0 with two; 8 groups of 512 rows 512 x 512 9.0,
// and 19.8 with two.)  Only the widths are gone through, not every count of tiles
// (2000 rows 8 x 113408: 100 us of host time per call, now 15).
struct GradientTiles {
  int64_t across;
  int32_t width, split;
};
GradientTiles gradient_tiles(int64_t rows, int32_t n, int64_t m_tiles, int64_t cols, int32_t box_cols) {
  const int64_t room[3] = {sm_count() / 2, clusters_at_once(2), clusters_at_once(4)}, pairs = room[0];
  const int64_t fewest = (cols + kTileN - 1) / kTileN;
  const int64_t blocks = (rows + 64 * n - 1) / (64 * static_cast<int64_t>(n));   // of an even group
  GradientTiles t = {0, 0, 1};
  int64_t best = INT64_MAX;
  for (int64_t w = kTileN; w > 0; w -= 32) {
    const int64_t across = (cols + w - 1) / w, even = (cols + across - 1) / across;
    if (across > 4 * fewest) break;
    for (int32_t i = 0; i < 3; ++i) {
      const int32_t s = 1 << i;
      const int64_t box = s == 1 ? box_cols : 32;
      if (w != (even + box - 1) / box * box || (s > 1 && (w > 128 || blocks < 4 * s))) continue;
      const int64_t tiles = m_tiles * across, each = std::max<int64_t>(w, 128) + 192;
      int64_t cost = split_cost(tiles, blocks, s, room[i], s == 1 ? 0 : s == 2 ? 17 : 25);
      if (cost == INT64_MAX) continue;
      cost = cost * each + (s == 1 ? (tiles + pairs - 1) / pairs * 10 * w : 0);   // (and a tile's way out)
      if (cost >= best) continue;
      best = cost;
      t = {across, static_cast<int32_t>(w), s};
    }
    if (m_tiles * t.across >= 6 * pairs) break;
  }
  return t;
}

// A launch's groups: all, those whose sums run in one piece, or those of several.
enum Groups { kAll, kShort, kLong };
template <int NOUT>
int gradient_launch(const himuon_mat *A, const himuon_mat *B, int32_t e0, int32_t n, const int32_t *offsets,
                    float alpha, float beta, const himuon_mat *C, int64_t c_stride, const himuon_mat *G,
                    int64_t g_stride, Groups groups, cudaStream_t stream) {
  MmaArgs<1, NOUT> a;
  common_args(a, offsets, e0, n, A->rows);
  const int64_t longest = (int64_t)1 << longest_log(G->dtype);
  const bool pieces = groups == kLong || G->dtype == HIMUON_FP32 || (groups == kAll && A->rows > longest);
  a.box_cols = pieces || (C && C->dtype == HIMUON_FP32) ? 32 : 64;
  const int64_t m_tiles = n * ((A->cols + kTileM - 1) / kTileM);
  const GradientTiles tiles = gradient_tiles(A->rows, n, m_tiles, B->cols, a.box_cols);
  const int64_t most = m_tiles * tiles.across;
  // Any group may have all the rows, as far as the host knows, but few need the
  // kernel of pieces, which has half the stages' length and narrower boxes: large
  // calls launch it for those alone (which costs 8 us where there is none).  fp16,
  // 64 groups 1024 x 4096: 32768 rows 299 us in one launch, 272 in two, 8192 rows 202
  // and 163; 32 groups 1024 x 2048, 1024 tiles, 97 and 98; 40 groups 768 x 768 25 and 30.
  if (groups == kAll && pieces && G->dtype != HIMUON_FP32 && tiles.split == 1 && A->rows <= n * longest &&
      most >= 16 * (sm_count() / 2)) {
    const int rc = gradient_launch<NOUT>(A, B, e0, n, offsets, alpha, beta, C, c_stride, G, g_stride, kShort, stream);
    return rc ? rc : gradient_launch<NOUT>(A, B, e0, n, offsets, alpha, beta, C, c_stride, G, g_stride, kLong, stream);
  }
  if (groups == kShort) a.most = static_cast<int32_t>(longest);
  if (groups == kLong) a.least = static_cast<int32_t>(longest) + 1;
  a.split = tiles.split;
  a.cap = tiles.width;
  a.mt_n = static_cast<int32_t>(tiles.across);
  if (A->rows == 0) {
    // no row is ever loaded: the maps only have to be valid, and G's memory is
    himuon_mat any = *G;
    any.dtype = A->dtype;
    any.rows = 1;
    any.cols = 8;
    if (!make_map(&a.w[0], any, 0, 0, 64)) return HIMUON_ERR_CUDA;
    a.x[0] = a.x[1] = a.x[2] = a.w[0];
  } else if (!make_map(&a.w[0], *A, 0, 0, 64) || !make_map(&a.x[0], *B, 0, 0, 64) ||
             !make_window_map(&a.x[1], *B) || !make_window_map(&a.x[2], *A)) {
    return HIMUON_ERR_CUDA;
  }
  a.K = 0;
  a.M = static_cast<int32_t>(A->cols);
  a.N = static_cast<int32_t>(B->cols);
  a.idesc = idesc_of(A->dtype, 1, 1);
  a.alpha = alpha;
  a.beta = beta;
  a.has_c = C != nullptr;
  a.mt_m = static_cast<int32_t>(m_tiles / n);
  if (a.split > 1) a.box_cols = 32;
  a.piece_log = piece_log(A->rows, a.split > 1 ? HIMUON_FP32 : G->dtype);
  for (int32_t i = 0; i < (NOUT > 1 ? n : 1); ++i) {
    if (!make_map(&a.g[i], G[e0 + i], NOUT > 1 ? 1 : n, g_stride, 32, a.box_cols)) return HIMUON_ERR_CUDA;
    a.out[i] = static_cast<char *>(G[e0 + i].data);
    if (C && !make_map(&a.c[i], C[e0 + i], NOUT > 1 ? 1 : n, c_stride, 32, a.box_cols)) return HIMUON_ERR_CUDA;
  }
  a.ldo = G->ld;
  a.out_stride = g_stride;
  a.odtype = G->dtype;
  if (C) a.cdtype = C->dtype;
  a.buffers = C && a.split == 1 ? 3 : 1;   // (a split tile's warps have one box each)
  if (a.split > 1) return launch_mma<0, 1, 1, 1, 1>(a, most, stream);
  return pieces ? launch_mma<0, 1, 1, 1, 0>(a, most, stream) : launch_mma<0, 1, 1, 0, 0>(a, most, stream);
}

}  // namespace

int expert_device() {
  const int rc = device_usable();
  if (rc) return rc;
  return load_kernels() ? HIMUON_OK : HIMUON_ERR_CUDA;
}

}  // namespace himuon

using namespace himuon;

extern "C" {

int himuon_expert_product(const himuon_mat *X, const himuon_mat *W, int32_t n, const int32_t *offsets, int32_t w_trans,
                          const himuon_mat *Y, void *stream) {
  if (!X || !W || !Y || n < 1 || n > kMaxGroups || (!offsets && n != 1) || (w_trans != 0 && w_trans != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (rc) return rc;
  if (!is16(X->dtype) || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->dtype != X->dtype || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if ((w_trans ? W->cols : W->rows) != X->cols || (w_trans ? W->rows : W->cols) != Y->cols) return HIMUON_ERR_INVALID;
  rc = expert_device();
  if (rc) return rc;
  return run_product(X, nullptr, W, nullptr, n, offsets, w_trans, Y, static_cast<cudaStream_t>(stream));
}

int himuon_expert_product_i8(const himuon_mat *X, const himuon_mat *x_scale, const himuon_mat *W,
                             const himuon_mat *w_scale, int32_t n, const int32_t *offsets, const himuon_mat *Y,
                             void *stream) {
  if (!X || !W || !Y || n < 1 || n > kMaxGroups || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (!rc) rc = check_scale(x_scale, 1, X->rows);
  if (!rc) rc = check_scale(w_scale, n, Y->cols);
  if (rc) return rc;
  if (X->dtype != HIMUON_I8 || W->dtype != HIMUON_I8 || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->cols != X->cols || W->rows != Y->cols || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if (X->cols > 131071) return HIMUON_ERR_UNSUPPORTED;   // 2^14 per term: the sum stays inside int32
  rc = expert_device();
  if (rc) return rc;
  return run_product(X, static_cast<const float *>(x_scale->data), W, w_scale, n, offsets, 1, Y,
                     static_cast<cudaStream_t>(stream));
}

int himuon_expert_gradient(const himuon_mat *A, const himuon_mat *B, int32_t n, const int32_t *offsets, float alpha,
                           float beta, const himuon_mat *C, const himuon_mat *G, void *stream) {
  if (!A || !B || !G || n < 1 || n > kMaxGroups || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  if (!isfinite(alpha) || !isfinite(beta) || (!C && beta != 0.f)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*A, 0);
  if (!rc) rc = check_operand(*B, 0);
  if (!rc) rc = check_list(G, n);
  if (!rc && C) rc = check_list(C, n);
  if (rc) return rc;
  if (!is16(A->dtype) || !is_float(G->dtype) || (C && !is_float(C->dtype))) return HIMUON_ERR_UNSUPPORTED;
  if (B->dtype != A->dtype || B->rows != A->rows || G->rows != A->cols || G->cols != B->cols) return HIMUON_ERR_INVALID;
  if (C && (C->rows != G->rows || C->cols != G->cols)) return HIMUON_ERR_INVALID;
  if (C && beta != 0.f && (C->ld != G->ld || C->dtype != G->dtype))
    for (int32_t e = 0; e < n; ++e)
      if (C[e].data == G[e].data) return HIMUON_ERR_INVALID;
  int64_t g_stride, c_stride = 0;
  const bool g_stacked = stacked(G, n, &g_stride);
  if (!g_stacked) {   // (stacked ones differ)
    std::vector<const void *> seen(n);
    for (int32_t e = 0; e < n; ++e) seen[e] = G[e].data;
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return HIMUON_ERR_INVALID;
  }
  rc = expert_device();
  if (rc) return rc;
  if (beta == 0.f) C = nullptr;
  const bool st = g_stacked && (!C || stacked(C, n, &c_stride));
  const int32_t cap = st ? kMaxStack : kMaxList;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t e0 = 0; e0 < n; e0 += cap) {
    const int32_t cnt = std::min(n - e0, cap);
    rc = st ? gradient_launch<1>(A, B, e0, cnt, offsets, alpha, beta, C, c_stride, G, g_stride, kAll, s)
            : gradient_launch<kMaxList>(A, B, e0, cnt, offsets, alpha, beta, C, 0, G, 0, kAll, s);
    if (rc) return rc;
  }
  return HIMUON_OK;
}

}  // extern "C"
