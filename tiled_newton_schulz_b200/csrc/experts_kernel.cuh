// experts_kernel.cuh -- the tcgen05 kernel behind the expert products and their
// weight gradients (included by experts.cu alone).
#pragma once
#include "experts.hpp"
#include "ptx.cuh"

namespace himuon {
namespace {

// One launch takes the matrices of up to kMaxStack groups when they lie at
// equal distances (one tensor map, or a base and a stride), else a list of up
// to kMaxList in the kernel's parameters; longer calls run as several
// launches, each on its own stretch of the offsets.
constexpr int kMaxStack = 256;

// ---------------------------------------------------------------- the product kernel
// Both directions are one tcgen05 product per output tile, D (256 x up to 256,
// fp32 or int32 in tensor memory) = A B^T over 128-byte stretches of K:
//   product:  A = W_e (256 channels), B = X (up to 256 rows of group e), so the
//             ragged side is the MMA's N, which is any multiple of 32: a group
//             of 5 rows costs a 32-column tile, not a 128-row one.
//   gradient: A = 256 columns of operand A, B = 256 columns of operand B,
//             K = the group's rows (both operands MN-major).
constexpr uint32_t kABytes = 16384;     // 128 rows (or 2 x 64 MN columns) x 128 bytes of K
constexpr uint32_t kBoxBytes = 2048;    // 16 rows of X x 128 bytes
constexpr uint32_t kData = 229376;      // operand ring and the epilogue's buffers
constexpr int kMaxStages = 10;
constexpr uint32_t kStageOut = 4096;    // an epilogue warp's buffer: 32 x 32 fp32, swizzled
constexpr int kEpiWarps = 8;
constexpr int kTileM = 256, kTileN = 256;   // a CTA pair's tile of D
constexpr int kThreads = 128 + 32 * kEpiWarps;   // three warpgroups: loads and MMAs (warps 0, 1), epilogue (4..11)
// Registers per thread of a kernel whose epilogue holds running sums: as launched,
// and after the loading warpgroup has given its own to the two of the epilogue.  A
// warpgroup that asks for more than the launch left over waits without an end, so
// the host refuses a build with fewer at launch (load_variant).
constexpr int kRegsLaunch = 168, kRegsLoad = 56, kRegsSums = 224;
static_assert(kRegsLoad + 2 * kRegsSums <= 3 * kRegsLaunch, "registers of the three warpgroups");
template <int GRAD, int PREC, int SPLIT>
constexpr bool kMovesRegisters = PREC && (GRAD || !SPLIT);   // the variants that do
// Sums of 16-bit operands: the tensor core's accumulator truncates at every K = 16
// step.  Terms of changing sign lose about 1e-8 of the result per step (K = 1100:
// 1.1e-6 against 2.6e-7 for rounded fp32 sums), terms of one sign 1e-7 (K = 2^22:
// 2.6%), which fits products cut at a quarter of the accumulator's last place and
// a sum cut at its last place: 2.5 places per step on average, 5 at most.  So long
// sums run in pieces of 2^piece_log elements, which the epilogue adds in fp32
// registers (PREC); the kernel without PREC is for sums of one piece.  2^12
// elements for fp16 results and 2^15 for bf16 keep 5 places per step below a third
// of a rounding to the type; fp32 results, and shared tiles, which have the sums in
// registers anyway, take 2^9 (K = 1100: 4.6e-7).  Every addition of a piece is off
// by 2^-24 of the sum so far, in one direction where the terms are equal, so beyond
// 2^20 elements the pieces grow with the root of the sum's length.
__host__ inline int32_t longest_log(int32_t dtype) {   // of a sum in one piece
  return dtype == HIMUON_FP32 ? 9 : dtype == HIMUON_FP16 ? 12 : 15;
}
__host__ inline int32_t piece_log(int64_t length, int32_t dtype) {
  int32_t log = longest_log(dtype);
  while (length > (1 << 20) && ((int64_t)1 << 2 * log) < 2 * length) ++log;
  return log;
}
constexpr uint32_t kBarBytes = 448;
constexpr uint32_t kSmem = kData + kBarBytes + 4 * (kMaxStack + 4) + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");

// NMAP, NOUT: tensor maps of W, and of G and C (the product writes Y without
// one): 1, over matrices at equal distances, or one for each of a list.
template <int NMAP, int NOUT>
struct MmaArgs {
  CUtensorMap w[NMAP];     // product: W; gradient: operand A
  // product: X in boxes of 128, 64, 32 and 16 rows; gradient: operand B, and the
  // windows (make_window_map) of B and A
  CUtensorMap x[4];
  const int32_t *offsets;
  int64_t rows;
  int32_t n;
  int32_t K;               // product: length of the sums
  int32_t M, N;            // product: M channels; gradient: G is M x N
  int32_t mt_m, mt_n;      // tiles along M; gradient: along N
  int32_t cap;             // gradient: columns of a tile (a multiple of 32); product: log2 of a tile's most rows
  int32_t split;           // pairs that share a tile's sum (the cluster's)
  int32_t piece_log;       // PREC: log2 of a piece's elements (whole stages)
  int32_t least, most;     // gradient: rows of the groups that the launch takes
  uint32_t idesc;          // without the N field
  int *status;
  const float *x_scale, *w_scale;
  int64_t ld_scale;
  CUtensorMap g[NOUT], c[NOUT];   // gradient: G and C in boxes of 32 rows x box_cols columns; product:
                                  // g[0], an fp32 Y in boxes of 16 rows x 32 columns
  char *out[NOUT];                // product: Y; gradient: G
  int64_t ldo, out_stride;        // (NOUT = 1: bytes between consecutive matrices of G)
  int32_t odtype, cdtype, has_c;
  int32_t buffers;                // of kStageOut per epilogue warp
  int32_t box_cols;               // 32, or 64 where G and C are 16-bit
  int32_t stall;                  // tests only: the first pair's MMA warp waits for what does not come
  float alpha, beta;
};

// Pair forms (CTA pairs, issued by the even CTA): both operands from shared
// memory at the same offsets in both CTAs.
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_i8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// TMA loads into this CTA's shared memory that complete on an mbarrier of
// either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int32_t x, int32_t y,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
// One thread of the converged warp (the same one every time).  The loops that
// issue copies and MMAs are run by whole warps, with only the instruction
// itself in the elected thread's branch: their addresses and descriptors then
// stay in uniform registers.  (Run by lane 0 alone, each stage's copies took
// about 500 cycles to issue and its MMAs 450, which bounded every case.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A bounded wait by a whole warp: its lanes agree on the outcome.  CLUSTER:
// for phases that the pair's other CTA also arrives on.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, int *status) {
  auto ready = [&] {
    return __all_sync(0xffffffffu, CLUSTER ? mbar_try_wait_cluster(bar, phase) : mbar_try_wait(bar, phase));
  };
  if (ready()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ready()) return true;
    if ((i & 255u) == 0 && __any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) break;
  }
  set_status(status, HIMUON_ERR_TIMEOUT_DEV);
  return false;
}

// Bound i of the groups, clamped into 0 .. rows.
__device__ __forceinline__ int32_t bound_at(const int32_t *offsets, int32_t i, int64_t rows) {
  if (!offsets) return i == 0 ? 0 : static_cast<int32_t>(rows);
  return static_cast<int32_t>(min(max((int64_t)offsets[i], (int64_t)0), rows));
}

__device__ __forceinline__ int32_t round32(int32_t x) { return (x + 31) / 32 * 32; }
// A group of cnt rows runs as ceil(cnt / 2^shift) tiles, its units of 32 rows
// (the pair's CTAs hold half of them each, in boxes of 16) dealt out as evenly
// as they go: tiles of equal width would pad up to 31 rows each (16381 rows of 61
// experts, 1024 -> 4096, a tenth of the MMAs' columns).
__device__ __forceinline__ int32_t row_tiles(int32_t cnt, int32_t shift) { return (cnt + (1 << shift) - 1) >> shift; }
__device__ __forceinline__ int32_t tile_width(int32_t cnt, int32_t shift) {   // the widest
  const int32_t mt = row_tiles(cnt, shift), units = (cnt + 31) / 32;
  return 32 * (mt <= 1 ? units : (units + mt - 1) / mt);
}

struct Tile {
  int32_t e;        // group
  int32_t m0;       // first row of D in the output: channel (product) or row of G
  int32_t n0;       // product: first row of X; gradient: first column of G
  int32_t width;    // columns of D: a multiple of 32
  int32_t valid;    // of them, inside the output
  int32_t k0, len;  // the sums' stretch: product, of K; gradient, rows (of the slice, where a tile is split)
};

// Tile `idx` of the launch: the same for the whole warp (ALONE), or each lane's own.
template <int GRAD, int SPLIT, int kElems, bool ALONE, typename Args>
__device__ __forceinline__ Tile tile_at(const Args &a, const int32_t *start, int32_t slice, int32_t idx) {
  Tile t;
  const uint32_t mt_m = a.mt_m, u = static_cast<uint32_t>(idx) / mt_m;
  if (GRAD) {
    const uint32_t i = u / static_cast<uint32_t>(a.mt_n);
    t.e = start[i];
    t.m0 = (idx - u * mt_m) * kTileM;
    t.n0 = (u - i * a.mt_n) * a.cap;
    t.valid = min(a.cap, a.N - t.n0);
    t.width = round32(t.valid);
    t.k0 = bound_at(a.offsets, t.e, a.rows);
    t.len = max(0, bound_at(a.offsets, t.e + 1, a.rows) - t.k0);
  } else {
    // the group whose row tiles hold row tile u: the last with start[e] <= u
    t.e = 0;
    if (ALONE) {
      for (const int lane = threadIdx.x & 31;; t.e += 32) {
        const int32_t e = t.e + 1 + lane;
        const uint32_t before = __ballot_sync(0xffffffffu, e < a.n && start[e] <= static_cast<int32_t>(u));
        if (before == 0xffffffffu) continue;
        t.e += __popc(before);
        break;
      }
    } else {
      for (int32_t end = a.n; end - t.e > 1;) {
        const int32_t mid = (t.e + end) / 2;
        if (start[mid] <= static_cast<int32_t>(u)) t.e = mid;
        else end = mid;
      }
    }
    const int32_t lo = bound_at(a.offsets, t.e, a.rows), hi = max(lo, bound_at(a.offsets, t.e + 1, a.rows));
    const int32_t cnt = hi - lo, mt = row_tiles(cnt, a.cap);
    // bands of up to 8 row tiles, row tile fastest: the tiles in flight share
    // a few panels of W and of X
    const uint32_t r = idx - start[t.e] * mt_m;
    const uint32_t g = mt <= 8 ? 0 : r / (8 * mt_m), rr = r - g * 8 * mt_m;
    const uint32_t gm = min(8, mt - 8 * static_cast<int32_t>(g)), mc = gm == 1 ? rr : rr / gm;
    const int32_t tt = 8 * g + rr - mc * gm;
    t.m0 = mc * kTileM;
    const int32_t units = (cnt + 31) / 32, each = mt <= 1 ? units : units / mt, more = units - each * mt;
    t.width = 32 * (each + (tt < more ? 1 : 0));
    t.n0 = lo + 32 * (tt * each + min(tt, more));
    t.valid = min(t.width, hi - t.n0);
    t.k0 = 0;
    t.len = a.K;
  }
  if (SPLIT) {   // this pair's blocks of the sum
    const int32_t nb = (t.len + kElems - 1) / kElems;
    const int32_t b0 = nb * slice / a.split, b1 = nb * (slice + 1) / a.split;
    t.k0 += b0 * kElems;
    t.len = min(t.len, b1 * kElems) - b0 * kElems;
  }
  return t;
}

// A role's tiles in order: first, first + step, ..  Finding one takes about 1200
// cycles of divisions and loads, a fifth of a tile of a short sum; so the lanes of
// the warp find one each, 32 tiles ahead, and hand them round.  A product's first
// one, which the launch waits for, is found by the whole warp.  (bf16, 7052 rows
// 128 -> 10968 55 -> 48 us, 16381 rows of 61 groups 1024 -> 4096 151 -> 148;
// gradients of 79 groups, 4688 rows, 4325 x 553, 235 -> 226; calls of a few tiles
// per pair are up to 2% slower.)
// AHEAD = 0: one at a time, where the registers are taken.
template <int GRAD, int SPLIT, int kElems, int AHEAD = 1>
struct Tiles {
  Tile own;
  int32_t taken = 0;
  template <typename Args>
  __device__ __forceinline__ Tile next(const Args &a, const int32_t *start, int32_t slice, int32_t idx, int32_t step,
                                       int32_t n_tiles) {
    const int lane = threadIdx.x & 31, from = taken & 31;
    if (!AHEAD || (!GRAD && idx < step)) return tile_at<GRAD, SPLIT, kElems, true>(a, start, slice, idx);
    ++taken;
    if (from == 0) {
      const int64_t mine = min(idx + int64_t(step) * lane, int64_t(n_tiles) - 1);
      own = tile_at<GRAD, SPLIT, kElems, false>(a, start, slice, static_cast<int32_t>(mine));
    }
    Tile t;
    t.e = __shfl_sync(0xffffffffu, own.e, from);
    t.m0 = __shfl_sync(0xffffffffu, own.m0, from);
    t.n0 = __shfl_sync(0xffffffffu, own.n0, from);
    t.valid = __shfl_sync(0xffffffffu, own.valid, from);
    t.width = GRAD ? round32(t.valid) : __shfl_sync(0xffffffffu, own.width, from);
    t.k0 = GRAD || SPLIT ? __shfl_sync(0xffffffffu, own.k0, from) : 0;
    t.len = GRAD || SPLIT ? __shfl_sync(0xffffffffu, own.len, from) : a.K;
    return t;
  }
};

// The product's output: 32 rows of Y x 32 channels, of which `rows` x `cols`
// are inside.  A lane comes with one channel of every row and leaves with runs
// of a row: the block is turned through the warp's buffer (16-byte chunk c of
// line r at chunk c ^ (r & 7): free of bank conflicts both ways), so that every
// row is written as one 64- or 128-byte run.  (A group's last rows end inside a
// tile, where a tensor map could not stop.)
template <typename T2>
__device__ __forceinline__ uint32_t two16(float x, float y);
template <>
__device__ __forceinline__ uint32_t two16<__half2>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t two16<__nv_bfloat162>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// 16-bit: line k holds rows 2 k and 2 k + 1, a 32-bit word per channel.
template <typename T2>
__device__ __forceinline__ void put_rows16(uint32_t *st, int lane, const float (&v)[32], uint16_t *out, int64_t ldo,
                                           int32_t rows, int32_t cols) {
  __syncwarp();   // the last block's readers are done
#pragma unroll
  for (int k = 0; k < 16; ++k)
    st[k * 32 + (((lane >> 2) ^ (k & 7)) << 2) + (lane & 3)] = two16<T2>(v[2 * k], v[2 * k + 1]);
  __syncwarp();
  const int32_t col = (lane & 3) * 8;
  uint16_t *o = out + (lane >> 2) * 2 * ldo + col;
#pragma unroll
  for (int p = 0; p < 2; ++p, o += 16 * ldo) {
    const int k = (lane >> 2) + 8 * p;
    const uint4 x = *reinterpret_cast<const uint4 *>(st + k * 32 + (((col >> 2) ^ (k & 7)) << 2));
    const uint4 y = *reinterpret_cast<const uint4 *>(st + k * 32 + ((((col >> 2) + 1) ^ (k & 7)) << 2));
    const uint4 a = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410),
                               __byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410));
    const uint4 b = make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632),
                               __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632));
    if (col + 8 <= cols) {
      if (2 * k < rows) *reinterpret_cast<uint4 *>(o) = a;
      if (2 * k + 1 < rows) *reinterpret_cast<uint4 *>(o + ldo) = b;
    } else {
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (col + j >= cols) break;
        if (2 * k < rows) o[j] = static_cast<uint16_t>(wa[j / 2] >> (16 * (j & 1)));
        if (2 * k + 1 < rows) o[ldo + j] = static_cast<uint16_t>(wb[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}
// fp32: line r holds row r.
__device__ __forceinline__ void put_rows32(float *st, int lane, const float (&v)[32], float *out, int64_t ldo,
                                           int32_t rows, int32_t cols) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 32; ++k) st[k * 32 + (((lane >> 2) ^ (k & 7)) << 2) + (lane & 3)] = v[k];
  __syncwarp();
  const int32_t col = (lane & 7) * 4;
  float *o = out + (lane >> 3) * ldo + col;
#pragma unroll
  for (int p = 0; p < 8; ++p, o += 4 * ldo) {
    const int r = (lane >> 3) + 4 * p;
    const float4 f = *reinterpret_cast<const float4 *>(st + r * 32 + (((col >> 2) ^ (r & 7)) << 2));
    if (r >= rows) continue;
    if (col + 4 <= cols) {
      *reinterpret_cast<float4 *>(o) = f;
    } else {
      const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < cols) o[j] = w[j];
    }
  }
}

// The gradient's epilogue buffers hold a box as TMA moves it: 32 rows of 128
// bytes (32 columns of fp32, 64 of 16 bits; 128-byte swizzle) or of 64 bytes (32
// columns of 16 bits; 64-byte swizzle).  A lane owns a row; both patterns are
// free of bank conflicts.  Chunk k (16 bytes) of this lane's row:
__device__ __forceinline__ uint32_t box_at(int lane, int k, bool wide) {
  return wide ? lane * 128 + ((k ^ (lane & 7)) << 4) : lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4);
}
// v = alpha v + beta (32 columns of this lane's row, from the box's chunk k0)
__device__ __forceinline__ void box_combine(const uint8_t *buf, int lane, int32_t dtype, int k0, bool wide, float alpha,
                                            float beta, float (&v)[32]) {
  if (dtype == HIMUON_FP32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 f = *reinterpret_cast<const float4 *>(buf + box_at(lane, k, true));
      v[4 * k] = fmaf(beta, f.x, alpha * v[4 * k]);
      v[4 * k + 1] = fmaf(beta, f.y, alpha * v[4 * k + 1]);
      v[4 * k + 2] = fmaf(beta, f.z, alpha * v[4 * k + 2]);
      v[4 * k + 3] = fmaf(beta, f.w, alpha * v[4 * k + 3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 u = *reinterpret_cast<const uint4 *>(buf + box_at(lane, k0 + k, wide));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 f = dtype == HIMUON_FP16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[h]))
                                              : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[h]));
        v[8 * k + 2 * h] = fmaf(beta, f.x, alpha * v[8 * k + 2 * h]);
        v[8 * k + 2 * h + 1] = fmaf(beta, f.y, alpha * v[8 * k + 2 * h + 1]);
      }
    }
  }
}
template <typename T2>
__device__ __forceinline__ void box_write16(uint8_t *buf, int lane, int k0, bool wide, const float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4 *>(buf + box_at(lane, k0 + k, wide)) =
        make_uint4(two16<T2>(v[8 * k], v[8 * k + 1]), two16<T2>(v[8 * k + 2], v[8 * k + 3]),
                   two16<T2>(v[8 * k + 4], v[8 * k + 5]), two16<T2>(v[8 * k + 6], v[8 * k + 7]));
}
__device__ __forceinline__ void box_write(uint8_t *buf, int lane, int32_t dtype, int k0, bool wide,
                                          const float (&v)[32]) {
  if (dtype == HIMUON_FP32) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4 *>(buf + box_at(lane, k, true)) =
          make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else if (dtype == HIMUON_FP16) {
    box_write16<__half2>(buf, lane, k0, wide, v);
  } else {
    box_write16<__nv_bfloat162>(buf, lane, k0, wide, v);
  }
}
// A box to memory by the warp, `rows` x `cols` of it: runs of 16 bytes, and single
// elements in the last column's run.
__device__ __forceinline__ void box_copy(const uint8_t *buf, int lane, int32_t dtype, int32_t box_cols, char *out,
                                         int64_t at, int64_t ld, int32_t rows, int32_t cols) {
  const int es = dtype == HIMUON_FP32 ? 4 : 2, per = 16 / es, runs = box_cols * es / 16;   // 4 or 8 runs per row
  const int run = lane % runs, have = min(per, cols - run * per);
  if (have <= 0) return;
  for (int r = lane / runs; r < rows; r += 32 / runs) {
    const uint4 u = *reinterpret_cast<const uint4 *>(buf + box_at(r, run, runs == 8));
    char *o = out + (at + r * ld + run * per) * es;
    if (have == per) {
      *reinterpret_cast<uint4 *>(o) = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= have) break;
        if (es == 4) reinterpret_cast<uint32_t *>(o)[j] = w[j & 3];
        else reinterpret_cast<uint16_t *>(o)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}
// fp32, whole rows: the block goes by TMA in two boxes of 16 rows (128-byte swizzle),
// from the buffer's halves in turn, turned without bank conflicts.  (7052 rows 128 -> 10968:
// 93 us with plain stores, 71 with boxes; 16-bit results gain nothing, 53.6 and 53.7.)
__device__ __forceinline__ void put_boxes32(const CUtensorMap *map, uint8_t *st, int lane, const float (&v)[32],
                                            int32_t x, int32_t y) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (elect_one()) bulk_wait_read<1>();   // this half has been read
    __syncwarp();
    uint8_t *box = st + 2048 * h;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      *reinterpret_cast<float *>(box + 128 * k + (((lane >> 2) ^ (k & 7)) << 4) + (lane & 3) * 4) = v[16 * h + k];
    fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
      tma_store_2d(map, box, x, y + 16 * h);
      bulk_commit();
    }
    __syncwarp();
  }
}

// The rows of group lane + 32 i (a whole warp, all loads in flight together).
// Reports offsets that decrease or leave 0 .. rows.
constexpr int kPerLane = kMaxStack / 32;
template <typename Args>
__device__ __forceinline__ void count_rows(const Args &a, int32_t (&cnt)[kPerLane], int lane) {
  int32_t o[kPerLane + 1];
#pragma unroll
  for (int i = 0; i <= kPerLane; ++i) {
    const int32_t e = lane + 32 * i;
    o[i] = e > a.n ? 0 : a.offsets ? a.offsets[e] : e == 0 ? 0 : static_cast<int32_t>(a.rows);
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    cnt[i] = 0;
    if (32 * i >= a.n) continue;
    const int32_t e = lane + 32 * i;
    const int32_t down = __shfl_down_sync(0xffffffffu, o[i], 1), over = __shfl_sync(0xffffffffu, o[i + 1], 0);
    const int64_t lo = o[i], hi = lane == 31 ? over : down;
    if (e < a.n) {
      if (lo < 0 || hi < lo || hi > a.rows) set_status(a.status, HIMUON_ERR_DEVICE);
      const int64_t first = min(max(lo, (int64_t)0), a.rows), last = min(max(hi, (int64_t)0), a.rows);
      cnt[i] = static_cast<int32_t>(max(last - first, (int64_t)0));
    }
  }
}

// The gradient's groups (a whole warp): those of least .. most rows, in order.
template <typename Args>
__device__ __forceinline__ void plan_groups(const Args &a, int32_t *list, int32_t *taken, int lane) {
  int32_t cnt[kPerLane];
  count_rows(a, cnt, lane);
  int32_t base = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    if (32 * i >= a.n) break;
    const bool mine = lane + 32 * i < a.n && cnt[i] >= a.least && cnt[i] <= a.most;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    if (mine) list[base + __popc(all & ((1u << lane) - 1))] = lane + 32 * i;
    base += __popc(all);
  }
  if (lane == 0) *taken = base;
}

// The product's tiles, from the groups' bounds (a whole warp): start[e], the
// row tiles of the groups before e, and the widest tile.
template <typename Args>
__device__ __forceinline__ void plan_rows(const Args &a, int32_t *start, int32_t *widest, int lane) {
  int32_t cnt[kPerLane];
  count_rows(a, cnt, lane);
  int32_t base = 0, w = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    if (32 * i >= a.n) break;
    w = max(w, tile_width(cnt[i], a.cap));
    int32_t s = row_tiles(cnt[i], a.cap);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    if (lane + 32 * i < a.n) start[lane + 32 * i + 1] = base + s;
    base += __shfl_sync(0xffffffffu, s, 31);
  }
  w = __reduce_max_sync(0xffffffffu, w);
  if (lane == 0) {
    start[0] = 0;
    *widest = w;
  }
}

// PREC: an epilogue warp's column groups half, half + 2, .. (below `in`) of
// accumulator piece p, added to its running sums.
template <int GROUPS>
__device__ __forceinline__ void read_pieces(float (&sum)[GROUPS][32], uint32_t taddr, int half, int32_t in,
                                            int32_t p, bool none) {
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const int32_t i = half + 2 * g;
    if (i >= in) continue;
    if (none) {
#pragma unroll
      for (int k = 0; k < 32; ++k) sum[g][k] = 0.f;
    } else if (p == 0) {
      tmem_ld32(taddr + 32 * i, sum[g]);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[16];
        tmem_ld16(taddr + 32 * i + 16 * h, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[g][16 * h + k] += v[k];
      }
    }
  }
}

// SPLIT: adds up the slices' sums of a tile.  Column group g of a warp belongs
// to the pair g % split; every pair's warp sends it its part over distributed
// shared memory, into the ring (free by then: the first cluster barrier follows
// every pair's last MMA), and the owner adds the parts in the order of the
// slices, whatever their order of arrival.  A warp has two groups at most and
// owns one: 4 KB per slice and warp, chunk k (16 bytes) of lane l at k * 512 + 16 l.
template <int GROUPS>
__device__ __forceinline__ void send_slices(float (&sum)[GROUPS][32], uint8_t *ring, int w, int lane, int half,
                                            int32_t in, int32_t rank, int32_t slice, int32_t split) {
  __syncwarp();
  cluster_sync_all();
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    if (half + 2 * g >= in) continue;
    const uint32_t part = smem_u32(ring + (slice * kEpiWarps + w) * kStageOut);
    const uint32_t to = mapa_shared(part, 2 * (g % split) + rank) + 16 * lane;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      st_cluster_v4(to + 512 * k, make_uint4(__float_as_uint(sum[g][4 * k]), __float_as_uint(sum[g][4 * k + 1]),
                                             __float_as_uint(sum[g][4 * k + 2]), __float_as_uint(sum[g][4 * k + 3])));
  }
  __syncwarp();
  cluster_sync_all();
}
// The total of the column group that the warp owns.
template <int KIND>
__device__ __forceinline__ void add_slices(float (&v)[32], const uint8_t *ring, int w, int lane, int32_t split) {
  const uint8_t *part = ring + w * kStageOut + 16 * lane;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int from = 0; from < 4; ++from) {
      if (from >= split) break;
      const float4 f = *reinterpret_cast<const float4 *>(part + from * kEpiWarps * kStageOut + 512 * k);
      const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float &t = v[4 * k + c];
        if (from == 0) t = x[c];
        else if (KIND) t = __int_as_float(__float_as_int(t) + __float_as_int(x[c]));
        else t += x[c];
      }
    }
  }
}

// KIND 0: 16-bit operands (kind::f16); 1: int8 (kind::i8).  A_MN: A is
// MN-major (W stored K x channels; the gradient's operands).  PREC: sums in
// pieces (piece_log); a product whose tiles are not shared then has an fp32 (1)
// or a 16-bit result (2): one kernel for both took 22.1 us for 1531 rows 1100 ->
// 2050 with an fp32 result, where this takes 21.7.
// SPLIT: the cluster's pairs share one tile, each a stretch of its sum (calls of
// few tiles of 128 columns at most); comes with PREC's running sums in registers.
//
// A pair of CTAs (cluster of 2) works on one 256-row tile of D: each CTA holds
// 128 of its rows (in its tensor memory) and of A's, and half of B's columns;
// the even CTA issues the MMAs for both.  A single CTA with the same 128 x 256
// tile writes and reads 96 + 96 bytes of operands per cycle of MMA in its
// shared memory, more than its 128 bytes per cycle; the pair needs 64 + 64.
// 8192 rows through 4096 -> 11008 take 468 to 495 us (1490 to 1580 TFLOP/s, the
// tensor pipe 91% active; at the power cap 556 us), 64 gradients of 1024 x 4096
// added in fp32 389 to 423 us (5.5 to 6.0 TB/s), 256 rows of 56 experts 84 to 87 us
// (5.4 to 5.6 TB/s).
// Persistent: warp 0 streams its CTA's operands through a ring of stages (TMA,
// completing on the even CTA's barriers), warp 1 of the even CTA issues each
// tile's MMAs into one of two accumulators, warps 4..11 of both drain the other
// one meanwhile.
template <int KIND, int A_MN, int GRAD, int NMAP, int NOUT, int PREC, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ MmaArgs<NMAP, NOUT> a) {
  constexpr int kElems = KIND ? 128 : 64;   // K elements per block of 128 bytes
  constexpr int kSub = GRAD && PREC && !SPLIT ? 1 : 2;   // blocks per stage
  constexpr int kStageK = kElems * kSub;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = kData - a.buffers * kEpiWarps * kStageOut;   // (a multiple of 1024)
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + kData);   // even CTA: both CTAs' loads
  uint64_t *empty = full + kMaxStages;        // each CTA: the stage's MMAs have read it
  uint64_t *acc_full = empty + kMaxStages;    // [2] each CTA: accumulator b holds a finished tile
  uint64_t *acc_empty = acc_full + 2;              // [2] even CTA: accumulator b drained by both CTAs
  uint64_t *drained = acc_empty + 2;               // [2] odd CTA: accumulator b drained by its warps
  uint64_t *done = drained + 2;                    // even CTA: every MMA issued has completed
  uint64_t *c_full = done + 1;                     // [3 per epilogue warp] a box of C has landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(c_full + 3 * kEpiWarps);
  int32_t *widest = reinterpret_cast<int32_t *>(tmem_slot + 1);   // product: columns of the widest tile; gradient: groups
  // product: [n + 1] the row tiles of the groups before; gradient: the groups of the launch
  int32_t *start = reinterpret_cast<int32_t *>(sm + kData + kBarBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kPieces = PREC && !KIND;   // (int32 sums are exact)
  constexpr int kGroups = !PREC ? 1 : SPLIT ? 2 : 4;   // PREC: 32-column groups of an epilogue warp's sums
  constexpr bool kMoved = kMovesRegisters<GRAD, PREC, SPLIT>;
  const int32_t piece = kPieces ? 1 << a.piece_log : 0;
  const int32_t cta = static_cast<int32_t>(cluster_ctarank());
  const int32_t rank = cta & 1, even = cta & ~1, slice = SPLIT ? cta >> 1 : 0;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << even);
  const int32_t ctas = SPLIT ? 2 * a.split : 2;
  const int32_t first = static_cast<int32_t>(blockIdx.x) / ctas, step = static_cast<int32_t>(gridDim.x) / ctas;
  grid_start_next();

  if (warp == 0) {
    // one barrier per lane and round: full, empty, acc_full, acc_empty, drained, done, c_full
    constexpr int kAcc = 2 * kMaxStages, kBars = kAcc + 7 + 3 * kEpiWarps;
    for (int i = lane; i < kBars; i += 32)
      mbar_init(full + i, i >= kAcc + 2 && i < kAcc + 4   ? kEpiWarps + 1
                          : i >= kAcc + 4 && i < kAcc + 6 ? kEpiWarps
                                                          : 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  grid_wait();   // nothing above reads or writes what earlier work of the stream does
  if (!GRAD && warp == 2) plan_rows(a, start, widest, lane);
  if (GRAD && warp == 2) plan_groups(a, start, widest, lane);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // barriers of both CTAs are ready before either is signalled
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int32_t all_tiles = (GRAD ? *widest * a.mt_n : start[a.n]) * a.mt_m;
  const int32_t n_tiles = SPLIT ? min(all_tiles, step) : all_tiles;   // (split: one tile per cluster)
  // a stage holds 128 rows of A and half of the widest tile's columns of B;
  // narrow tiles (few rows per expert) get more stages, so that enough of W is
  // in flight
  const uint32_t b_bytes =
      GRAD ? (a.cap / 2 + 63) / 64 * 8192u : (*widest + 31) / 32 * kBoxBytes;
  const uint32_t block_bytes = (kABytes + b_bytes + 1023) / 1024 * 1024, stage_bytes = kSub * block_bytes;
  const int stages = min(static_cast<int>(ring / stage_bytes), kMaxStages);

  // The three warpgroups take their roles here.  PREC: the epilogue's running sums
  // take 128 registers per thread, so 3 x 168 per thread become 56 + 2 x 224
  // (kRegsLoad, kRegsSums): one instruction for a whole warpgroup, as setmaxnreg
  // asks, ahead of any branch between its warps.
  if (warp < 4) {
    if (kMoved) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), even);
      int s = 0;
      uint32_t phase = 1;   // parity of the stage's last release; the first round finds it free
      bool ok = true;
      int64_t issued = 0;
      Tiles<GRAD, SPLIT, kElems, !SPLIT && !(GRAD && PREC)> tiles;
      Tile t, next;
      if (first < n_tiles) next = tiles.next(a, start, slice, first, step, n_tiles);
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        t = next;
        const bool more = idx + step < n_tiles;   // the next tile is looked up behind this one's first block
        if (more && t.len == 0) next = tiles.next(a, start, slice, idx + step, step, n_tiles);
        const int32_t len = t.len;
        const CUtensorMap *mw = NMAP > 1 ? &a.w[t.e] : &a.w[0];
        const int32_t z = NMAP > 1 ? 0 : t.e;
        const int32_t half = t.width / 2;
        const int32_t m0 = t.m0 + 128 * rank, n0 = t.n0 + half * rank;
        const int32_t boxes = GRAD ? (half + 63) / 64 : half / 16;
        const uint32_t bytes = kABytes + boxes * (GRAD ? 8192u : kBoxBytes);
        for (int32_t k = 0; k < len; k += kStageK) {
          if (!(ok = warp_wait(empty + s, phase, a.status))) break;
          uint8_t *As = sm + s * stage_bytes, *Bs = As + kABytes;
          const uint32_t bar = full0 + 8 * s;
          if (GRAD) {
            // a group's last rows, fewer than a block: they go to the block's end,
            // behind rows of zeros (rows -(64 - left) .. of their window), so that
            // no row of another group, whatever it holds, meets the MMAs
            if (elect_one()) {
              const bool both = kSub > 1 && k + kElems < len;
              if (rank == 0) mbar_arrive_expect_tx(full + s, both ? 4 * bytes : 2 * bytes);
  #pragma unroll
              for (int u = 0; u < kSub; ++u) {
                if (u > 0 && !both) break;
                uint8_t *Au = As + u * block_bytes, *Bu = Bs + u * block_bytes;
                const int32_t y = t.k0 + k + u * kElems, left = len - k - u * kElems;
                if (left < kElems) {
                  tma_load_3d_pair(Au, &a.x[2], m0, left - kElems, y, bar);
                  tma_load_3d_pair(Au + 8192, &a.x[2], m0 + 64, left - kElems, y, bar);
                  tma_load_3d_pair(Bu, &a.x[1], n0, left - kElems, y, bar);
                  if (boxes > 1) tma_load_3d_pair(Bu + 8192, &a.x[1], n0 + 64, left - kElems, y, bar);
                } else {
                  tma_load_2d_pair(Au, &a.w[0], m0, y, bar);
                  tma_load_2d_pair(Au + 8192, &a.w[0], m0 + 64, y, bar);
                  tma_load_2d_pair(Bu, &a.x[0], n0, y, bar);
                  if (boxes > 1) tma_load_2d_pair(Bu + 8192, &a.x[0], n0 + 64, y, bar);
                }
              }
            }
          } else if (elect_one()) {
            const bool both = kSub > 1 && k + kElems < len;
            if (rank == 0) mbar_arrive_expect_tx(full + s, both ? 4 * bytes : 2 * bytes);
  #pragma unroll
            for (int u = 0; u < kSub; ++u) {
              if (u > 0 && !both) break;
              uint8_t *Au = As + u * block_bytes, *Bu = Bs + u * block_bytes;
              const int32_t ku = t.k0 + k + u * kElems;
              if (A_MN) {
                tma_load_3d_pair(Au, mw, m0, ku, z, bar);
                tma_load_3d_pair(Au + 8192, mw, m0 + 64, ku, z, bar);
              } else {
                tma_load_3d_pair(Au, mw, ku, m0, z, bar);
              }
              // this CTA's rows of the tile in at most four boxes, the largest first
              int32_t at = 0;
  #pragma unroll
              for (int32_t i = 0; i < 4; ++i)
                if (boxes & (8 >> i)) {
                  tma_load_2d_pair(Bu + kBoxBytes * at, &a.x[i], ku, n0 + 16 * at, bar);
                  at += 8 >> i;
                }
            }
          }
          __syncwarp();
          if (k == 0 && more) next = tiles.next(a, start, slice, idx + step, step, n_tiles);
          ++issued;
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // the last loads have landed before the CTA ends, also when something gave
      // up (the even CTA's barriers see both CTAs' loads; the CTAs leave together)
      if (rank == 0)
        for (int64_t i = max((int64_t)0, issued - stages); i < issued; ++i)
          warp_wait(full + i % stages, static_cast<uint32_t>((i / stages) & 1), a.status);
    } else if (warp == 1) {
      if (rank == 0) {
        // descriptors of stage 0, without the address
        const uint64_t a_bits = A_MN ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024);
        const uint64_t b_bits = GRAD ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024);
        constexpr uint32_t kStepA = (A_MN ? 2048 : 32) >> 4, kStepB = (GRAD ? 2048 : 32) >> 4;
        int s = 0;
        uint32_t phase = 0;
        int32_t j = 0;
        bool ok = !a.stall || blockIdx.x != 0 || warp_wait(done, 0, a.status);
        Tiles<GRAD, SPLIT, kElems, !SPLIT && !(GRAD && PREC)> tiles;
        Tile t, next;
        if (first < n_tiles) next = tiles.next(a, start, slice, first, step, n_tiles);
        for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
          t = next;
          const bool more = idx + step < n_tiles;
          if (more && t.len == 0) next = tiles.next(a, start, slice, idx + step, step, n_tiles);
          const int32_t len = t.len;
          const uint32_t idesc = a.idesc | (static_cast<uint32_t>(t.width >> 3) << 17);
          uint32_t d = 0;
          // the next accumulator, once the epilogue has drained it
          auto acquire = [&] {
            const int b = j & 1;
            d = tmem + static_cast<uint32_t>(b * kTileN);
            const uint32_t parity = static_cast<uint32_t>(((j >> 1) - 1) & 1);
          const bool free = j < 2 || warp_wait<true>(acc_empty + b, parity, a.status);
            tc_fence_after();
            return free;
          };
          auto hand_over = [&] {
            if (elect_one()) mma_commit_pair(acc_full + (j & 1), pair_mask);
            __syncwarp();
            ++j;
          };
          if (len == 0) {
            if (!(ok = acquire())) break;
            hand_over();
          }
          for (int32_t k = 0; k < len; k += kStageK) {
            const uint32_t as = smem_u32(sm) + s * stage_bytes;
            const int32_t left = len - k;
            const bool fresh = kPieces ? (k & (piece - 1)) == 0 : k == 0;
            if (fresh && !(ok = acquire())) break;
            if (!(ok = warp_wait(full + s, phase, a.status))) break;
            tc_fence_after();
            // (a shared-memory address carries the CTA's rank above the descriptor's field)
            const uint64_t ad = a_bits | ((as >> 4) & 0x3FFF), bd = b_bits | (((as + kABytes) >> 4) & 0x3FFF);
            const int32_t begin = GRAD ? (kElems - min(left, kElems)) / 16 : 0;
            if (elect_one()) {
  #pragma unroll
              for (int32_t kk = 0; kk < 4 * kSub; ++kk) {
                // 16 (int8: 32) elements of K at a time; of a block that is not
                // full, the product's lie at its start, the gradient's at its end
                if (kk > 0 && (GRAD ? kk / 4 * kElems : kk * (kElems / 4)) >= left) break;
                if (GRAD && kk % 4 < (kElems - min(left - kk / 4 * kElems, kElems)) / 16) continue;
                const uint32_t off = (kk / 4) * (block_bytes >> 4);
                const uint64_t au = ad + off + (kk % 4) * kStepA, bu = bd + off + (kk % 4) * kStepB;
                const uint32_t add = !fresh || kk > begin ? 1u : 0u;
                if (KIND) mma_i8_ss_pair(d, au, bu, idesc, add);
                else mma_ss_pair(d, au, bu, idesc, add);
              }
              mma_commit_pair(empty + s, pair_mask);   // the stage is free in both CTAs once these MMAs have read it
            }
            __syncwarp();
            if (left <= kStageK || (kPieces && ((k + kStageK) & (piece - 1)) == 0)) hand_over();
            if (k == 0 && more) next = tiles.next(a, start, slice, idx + step, step, n_tiles);
            if (++s == stages) {
              s = 0;
              phase ^= 1;
            }
          }
        }
        // nothing is in flight when the pair leaves and releases its tensor memory
        if (elect_one()) mma_commit_pair(done, static_cast<uint16_t>(1u << even));
        __syncwarp();
        warp_wait(done, 0, a.status);
      }
    } else if (warp == 3 && rank == 1) {
      // Passes the odd CTA's "drained" on to the even one.  An arrival there
      // waits for the thread's earlier stores to be performed (cluster scope,
      // 1 to 2.5 thousand cycles beside a tile's stores); the epilogue's warps
      // arrive in their own CTA instead.
      const uint32_t free0 = mapa_shared(smem_u32(acc_empty), even);
      Tiles<GRAD, SPLIT, kElems, !SPLIT && !(GRAD && PREC)> tiles;
      int32_t j = 0;
      bool ok = true;
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        const int32_t len = GRAD || SPLIT ? tiles.next(a, start, slice, idx, step, n_tiles).len : a.K;
        const int32_t pieces = kPieces ? max(1, (len + piece - 1) >> a.piece_log) : 1;
        for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
          const int b = j & 1;
          ok = warp_wait(drained + b, static_cast<uint32_t>((j >> 1) & 1), a.status);
          tc_fence_after();
          tc_fence_before();
          if (ok && elect_one()) mbar_arrive_cluster(free0 + 8 * b);
          __syncwarp();
        }
      }
    }
  } else {
    if (kMoved) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
    if (GRAD) {
      // This warp's boxes of G, 32 rows x 32 or 64 columns, in the order of its tiles
      // and, inside one, of the columns.  With C, the boxes of C come by TMA up
      // to two ahead of the one at work, also from the next tile, and the result
      // takes their place: three buffers, so that a buffer is loaded again one
      // box after its store was issued.
      const int q = warp & 3;             // TMEM lanes 32 q .. 32 q + 31
      const int half = (warp - 4) >> 2;   // the warp's column groups: half, half + 2, .. (split: its slice's)
      const int32_t i0 = SPLIT ? half + 2 * slice : half, di = SPLIT ? 2 * a.split : 2;
      const int32_t bc = PREC ? 32 : a.box_cols;
      uint8_t *buf = sm + ring + (warp - 4) * a.buffers * kStageOut;
      uint64_t *landed = c_full + 3 * (warp - 4);
      uint64_t *freed = rank == 0 ? acc_empty : drained;
      const uint32_t c_bytes = bc * (a.cdtype == HIMUON_FP32 ? 128 : 64);
      // A box that reaches over the last column is stored up to the end of that
      // column's 16 bytes (observed: columns behind it in the row's pitch were
      // overwritten); where G's width is no multiple of 16 bytes the warp copies
      // the last boxes itself.
      const bool whole_runs = a.N % (a.odtype == HIMUON_FP32 ? 4 : 8) == 0;
      Tiles<GRAD, SPLIT, kElems, !PREC> tiles, c_tiles;   // at work; C's boxes
      struct Box {
        int32_t idx, i;   // tile, column group; idx >= n_tiles: none left
        Tile t;
      };
      auto groups = [&](const Tile &t) {   // of this tile that are inside G
        return t.m0 + 128 * rank + 32 * q < a.M ? (t.valid + bc - 1) / bc : 0;
      };
      auto settle = [&](Box &x) {   // to the first box at or after (idx, i)
        while (x.idx < n_tiles && x.i >= groups(x.t)) {
          x.idx += step;
          x.i = i0;
          if (x.idx < n_tiles) x.t = c_tiles.next(a, start, slice, x.idx, step, n_tiles);
        }
      };
      auto load_c = [&](Box &x, int at) {   // box x into buffer `at`, then on to the next box
        if (x.idx >= n_tiles) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(landed + at, c_bytes);
          tma_load_3d(buf + at * kStageOut, NOUT > 1 ? &a.c[x.t.e] : &a.c[0], x.t.n0 + bc * x.i,
                      x.t.m0 + 128 * rank + 32 * q, NOUT > 1 ? 0 : x.t.e, landed + at);
        }
        __syncwarp();
        x.i += di;
        settle(x);
      };
      Box ahead{first, i0, {}};
      if (a.has_c && first < n_tiles) {
        ahead.t = c_tiles.next(a, start, slice, first, step, n_tiles);
        settle(ahead);
        load_c(ahead, 0);
        load_c(ahead, 1);
      }
      int at = 0;                  // buffer of the box at work
      uint32_t c_phase = 0;        // per buffer
      bool ok = true;
      int32_t j = 0;
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        const Tile t = tiles.next(a, start, slice, idx, step, n_tiles);
        const int32_t in = groups(t);
        // column group i: combine with C, store.  fetch(h, v): its 32-column
        // part h from the accumulator or the running sums.
        auto emit = [&](int32_t i, auto fetch) {
          const int32_t m = t.m0 + 128 * rank + 32 * q, n0 = t.n0 + bc * i;
          const bool by_box = n0 + bc <= a.N || whole_runs;
          uint8_t *box = buf + at * kStageOut;
          float v[32];
          fetch(0, v);
          if (a.has_c) {
            if (!(ok = warp_wait(landed + at, (c_phase >> at) & 1, a.status))) return;
            c_phase ^= 1u << at;
          } else {
            if (elect_one()) bulk_wait_read<0>();   // (the last box's store has read the buffer)
            __syncwarp();
          }
  #pragma unroll
          for (int h = 0; h < (PREC ? 1 : 2); ++h) {
            if (32 * h >= bc) break;
            if (h > 0) fetch(h, v);
            if (a.has_c) {
              box_combine(box, lane, a.cdtype, 4 * h, bc == 64, a.alpha, a.beta, v);
              if (bc == 32) __syncwarp();   // (G's rows may lie where C's of other lanes did)
            } else {
  #pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= a.alpha;
            }
            box_write(box, lane, a.odtype, 4 * h, bc == 64, v);
          }
          if (!by_box) {
            __syncwarp();
            box_copy(box, lane, a.odtype, bc, (NOUT > 1 ? a.out[t.e] : a.out[0] + t.e * a.out_stride), m * a.ldo + n0,
                     a.ldo, min(32, a.M - m), a.N - n0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            if (by_box) tma_store_3d(NOUT > 1 ? &a.g[t.e] : &a.g[0], box, n0, m, NOUT > 1 ? 0 : t.e);
            bulk_commit();
            if (a.has_c) bulk_wait_read<1>();   // the store of the box before has read its buffer
          }
          __syncwarp();
          if (a.has_c) load_c(ahead, at == 0 ? 2 : at - 1);
          at = at + 1 == a.buffers ? 0 : at + 1;
        };
        const int32_t pieces = kPieces ? max(1, (t.len + piece - 1) >> a.piece_log) : 1;
        float sum[kGroups][32];
        for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
          const int b = j & 1;
          if (!(ok = warp_wait(acc_full + b, static_cast<uint32_t>((j >> 1) & 1), a.status))) break;
          tc_fence_after();
          const uint32_t taddr = tmem + static_cast<uint32_t>(b * kTileN) + (static_cast<uint32_t>(q * 32) << 16);
          auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(freed + b);
          };
          if (PREC && (SPLIT || pieces > 1)) {
            read_pieces(sum, taddr, half, in, p, SPLIT && t.len == 0);   // (several pieces: not empty)
            release();
            if (!SPLIT && p + 1 == pieces) {
  #pragma unroll
              for (int g = 0; g < kGroups; ++g)
                if (half + 2 * g < in && ok)
                  emit(half + 2 * g, [&](int, float(&v)[32]) {
  #pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = sum[g][k];
                  });
            }
          } else {
            for (int32_t i = half; i < in && ok; i += 2) {
              emit(i, [&](int h, float(&v)[32]) {
                if (t.len == 0) {
  #pragma unroll
                  for (int k = 0; k < 32; ++k) v[k] = 0.f;
                } else {
                  tmem_ld32(taddr + bc * i + 32 * h, v);
                  tmem_wait_ld();
                }
                if (i + 2 >= in && 32 * (h + 1) >= bc) release();   // the accumulator is read
              });
            }
            if (in <= half) release();   // no box of this warp's in the tile
          }
        }
        if (SPLIT) {
          send_slices(sum, sm, warp - 4, lane, half, in, rank, slice, a.split);
          if (half + 2 * slice < in && ok)
            emit(half + 2 * slice, [&](int, float(&v)[32]) { add_slices<KIND>(v, sm, warp - 4, lane, a.split); });
        }
      }
      if (SPLIT && first >= n_tiles) {   // the cluster has no tile: keep step with its barriers
        cluster_sync_all();
        cluster_sync_all();
      }
      if (!ok && a.has_c) {   // gave up: what was loaded ahead lands before the CTA ends (bounded)
        for (int k = 0; k < a.buffers; ++k) warp_wait(landed + k, (c_phase >> k) & 1, a.status);
      }
      if (elect_one()) bulk_wait0();
    } else {
      const int q = warp & 3;             // TMEM lanes 32 q .. 32 q + 31
      const int half = (warp - 4) >> 2;   // the warp's 32-column groups: half, half + 2, ..
      float *st = reinterpret_cast<float *>(sm + ring + (warp - 4) * kStageOut);
      uint64_t *freed = rank == 0 ? acc_empty : drained;
      const bool whole_runs = a.M % 4 == 0;   // (a box stores 16 bytes at a time)
      int32_t j = 0;
      Tiles<GRAD, SPLIT, kElems, !PREC> tiles;
      bool ok = true;
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        const Tile t = tiles.next(a, start, slice, idx, step, n_tiles);
        const int32_t m = t.m0 + 128 * rank + 32 * q;   // this warp's 32 channels
        const int32_t m_in = min(32, a.M - m);
        float chan = 1.f;
        if (KIND && lane < m_in) chan = a.w_scale[t.e * a.ld_scale + m + lane];
        const int32_t in = m_in > 0 ? (t.valid + 31) / 32 : 0;
        auto emit = [&](int32_t i, float(&v)[32]) {   // rows 32 i .. of the tile
          const int64_t r0 = t.n0 + 32 * i;
          const int32_t r_in = min(32, t.valid - 32 * i);
          if (KIND) {   // int32 sums: scales of this lane's channel and of each row
            const float mine = lane < r_in ? a.x_scale[r0 + lane] : 0.f;
  #pragma unroll
            for (int k = 0; k < 32; ++k)
              v[k] = static_cast<float>(__float_as_int(v[k])) * chan * __shfl_sync(0xffffffffu, mine, k);
          }
          const int64_t o = r0 * a.ldo + m;
          if (PREC != 2 && ((PREC && !SPLIT) || a.odtype == HIMUON_FP32)) {
            if (r_in == 32 && (m_in == 32 || whole_runs)) {
              put_boxes32(&a.g[0], reinterpret_cast<uint8_t *>(st), lane, v, m, static_cast<int32_t>(r0));
            } else {   // a box would reach the next group's rows, or 16 bytes into the padding
              if (elect_one()) bulk_wait_read<0>();
              put_rows32(st, lane, v, reinterpret_cast<float *>(a.out[0]) + o, a.ldo, r_in, m_in);
            }
          } else if (a.odtype == HIMUON_FP16)
            put_rows16<__half2>(reinterpret_cast<uint32_t *>(st), lane, v, reinterpret_cast<uint16_t *>(a.out[0]) + o,
                                a.ldo, r_in, m_in);
          else
            put_rows16<__nv_bfloat162>(reinterpret_cast<uint32_t *>(st), lane, v,
                                       reinterpret_cast<uint16_t *>(a.out[0]) + o, a.ldo, r_in, m_in);
        };
        const int32_t pieces = kPieces ? (t.len + piece - 1) >> a.piece_log : 1;
        float sum[kGroups][32];
        for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
          const int b = j & 1;
          if (!(ok = warp_wait(acc_full + b, static_cast<uint32_t>((j >> 1) & 1), a.status))) break;
          tc_fence_after();
          const uint32_t taddr = tmem + static_cast<uint32_t>(b * kTileN) + (static_cast<uint32_t>(q * 32) << 16);
          if (PREC && (SPLIT || pieces > 1)) {
            read_pieces(sum, taddr, half, in, p, false);
          } else {
  #pragma unroll 1
            for (int32_t i = half; i < in; i += 2) {
              tmem_ld32(taddr + 32 * i, sum[0]);
              tmem_wait_ld();
              emit(i, sum[0]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (elect_one()) mbar_arrive(freed + b);
          if (PREC && !SPLIT && pieces > 1 && p + 1 == pieces) {
  #pragma unroll
            for (int g = 0; g < kGroups; ++g)
              if (half + 2 * g < in) emit(half + 2 * g, sum[g]);
          }
        }
        if (SPLIT) {
          send_slices(sum, sm, warp - 4, lane, half, in, rank, slice, a.split);
          if (half + 2 * slice < in) {
            float v[32];
            add_slices<KIND>(v, sm, warp - 4, lane, a.split);
            emit(half + 2 * slice, v);
          }
        }
      }
      if (SPLIT && first >= n_tiles) {   // the cluster has no tile: keep step with its barriers
        cluster_sync_all();
        cluster_sync_all();
      }
      if (elect_one()) bulk_wait0();
    }
  }
  if (SPLIT && warp < 4) {   // the two barriers of send_slices
    __syncwarp();
    cluster_sync_all();
    cluster_sync_all();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // the pair leaves together: neither's memory goes while the other may signal or read it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

}  // namespace
}  // namespace himuon
